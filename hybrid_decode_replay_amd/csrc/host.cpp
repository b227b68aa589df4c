// host.cpp -- the C ABI (include/replayssm.h): validation, state layout,
// phase tracking, kernel selection and launch.  No call synchronizes.
#include "../../include/replayssm.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

#include "internal.hpp"
#include "kv.hpp"

namespace rs {

// Rows that share a key/value head fill 16-row products.  Up to 32 rows a wave takes one or two such
// blocks and the waves of a workgroup split the tokens; past that the cache goes through LDS and the
// waves take different rows.  Wide heads have one block a wave there (registers).  More rows than a
// workgroup holds make further chunks, which read the cache again (128 channels, 128 rows 155 us, 256 rows in
// two chunks 264).
KvPlan kv_attention_plan(int D, bool fp8, int rows)
{
    KvPlan p;
    p.wide = rows > 32;
    p.RB = rows <= 16 || (p.wide && D == 256) ? 1 : 2;
    p.RW = p.wide ? (rows > 64 || D == 256 ? 4 : 2) : 1;
    const int most = 16 * p.RB * p.RW;
    p.rpc = rows < most ? rows : most;
    p.nchunk = (rows + most - 1) / most;
    p.nwg = 256 * (p.wide ? 2 : kv_occ(D, fp8, p.RB));
    return p;
}

// Whether each range takes a workgroup of its own, with nothing to join, from what the host knows: the
// most tokens a range can have (the table's or the window's), not the lengths.  Times in us:
//   alone   the longest range in one workgroup.  A workgroup reads 40 GB/s (256 bytes a token 6.6 us per
//           1024 tokens, 512 bytes 12.4, 1024 bytes 25); through LDS it is the work that counts, 21 us per
//           1024 tokens of 128 channels and 42 of 256, for E4M3 too.
//   join    what a split adds: the second launch, and its rows (one range 5 us on the device, 192 ranges of
//           4 rows 6, of 32 rows 15, of 64 rows 24), and up to 2.5 us of the host's, which is what small
//           calls wait for that are not captured.
//   even    what a split takes at least: a tile in each workgroup, or all ranges at the chip's rate.
// The rows and the third count up to 20 and 8 us, since ranges may be much shorter than they can be, and the
// chip then waits for the one that is not.
// Measured with a cold cache, whole / split: one range of 256 tokens 5.9 / 10.1 (D 64), 8.9 / 11.6 (128), 13.4 /
// 14.9 (256), of 1024 11.0 / 10.3, 18.2 / 11.7, 32 / 15; 192 ranges of 2048 tokens 24.0 / 28.5, 41 / 44, 77 / 76,
// with 32 rows of a head 26.5 / 41.4, 45 / 57, 85 / 103; 504 ranges of up to 2048 tokens (D 64) 37 / 45, one of
// 2048 among others of 128 21 / 17.  Over 1037 such calls (widths, types, 4 to 128 rows, 1 to 6400 ranges; even
// lengths, a ramp, one long one) the rule costs 2, 5 and 8 % against the better choice, 1.9 times at worst;
// limits of tokens alone cost 5, 8 and 9, and 2.5 times.  What the lengths themselves say is weighed in
// the kernel where there are more ranges than workgroups (kv_order).
bool kv_attention_whole(const KvPlan& p, int D, bool fp8, long long tokens, long long ranges)
{
    const double bytes = 2.0 * D * (fp8 ? 1 : 2), token = p.wide ? 160e-6 * D : bytes / 40e3;
    const double alone = tokens * token, split = (double)(ranges < p.nwg ? ranges : p.nwg);
    const double rows = split * p.rpc / 400, join = 7.5 + (rows < 20 ? rows : 20);
    const double all = ranges * tokens * bytes / 5.9e6, even = all < 8 ? all : 8, tile = 128 * token;
    return ranges < (1 << 22) && alone <= join + (even > tile ? even : tile);
}

}  // namespace rs

struct replay_state {
    replay_config cfg;
    uint8_t* mem;
    size_t bytes;
    replay_layout lay;
    int parity;   // bookkeeping copy that holds the current values
    int phase;    // 0 idle, 1 drafts pending
    replay_stack* stack = nullptr;   // set while bound to a stack (which then owns the bookkeeping)
    bool needs_load = false;         // a former stack member: its own bookkeeping is stale
};

// Layers of one model share one bookkeeping set (layer 0's region).  A model
// step runs every layer once, in order; `next` is the layer it expects.
struct replay_stack {
    std::vector<replay_state*> layers;
    int32_t* book;
    uint32_t* err;
    int parity = 0;
    int phase = 0;    // 0 idle, 1 drafts pending
    int next = 0;     // next layer of the current step (0 between steps)
    int step_mode = -1;
    int step_k = 0;
    const uint8_t* step_active = nullptr;   // the active mask every layer of the step uses
};

namespace {

thread_local std::string g_err;

replay_status fail(replay_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
replay_status fail(replay_status s, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return s;
}

replay_status ok()
{
    g_err.clear();
    return REPLAY_OK;
}

replay_status hip_check(hipError_t e, const char* what)
{
    if (e != hipSuccess) return fail(REPLAY_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

// Clears an error an earlier, unrelated HIP call may have left behind, so that
// the hipGetLastError a launcher returns reports its own launch only.
hipError_t fresh() { return hipGetLastError(); }

// hip_check of a launch expression, after clearing any stale error (the comma
// operator sequences the clearing before the launch).
#define LAUNCH(expr, what) hip_check(((void)fresh(), (expr)), what)

rs::SlotMap all_tiles(int H)
{
    rs::SlotMap m;
    m.n = 0;
    m.H = H;
    return m;
}

uint64_t align256(uint64_t x) { return (x + 255) & ~(uint64_t)255; }

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int io_bytes(const replay_config* c) { return c->io_dtype == REPLAY_BF16 ? 2 : 4; }
int ckpt_bytes(const replay_config* c)
{
    return c->ckpt_dtype == REPLAY_F16 ? 2 : (c->ckpt_dtype == REPLAY_FP8_E4M3 ? 1 : 4);
}
int ck_kind(const replay_config* c)
{
    return c->ckpt_dtype == REPLAY_F16 ? rs::CK_F16 : (c->ckpt_dtype == REPLAY_FP8_E4M3 ? rs::CK_FP8 : rs::CK_F32);
}

replay_status check_config(const replay_config* c)
{
    if (!c) return fail(REPLAY_ERR_ARG, "config is NULL");
    if (c->abi_version != REPLAY_ABI_VERSION)
        return fail(REPLAY_ERR_ARG, "abi_version %d, library implements %d", c->abi_version, REPLAY_ABI_VERSION);
    if (c->kind != REPLAY_MAMBA2 && c->kind != REPLAY_GDN) return fail(REPLAY_ERR_ARG, "unknown kind %d", c->kind);
    if (c->batch < 1 || c->nheads < 1 || c->ngroups < 1)
        return fail(REPLAY_ERR_SHAPE, "batch, nheads and ngroups must be >= 1");
    if (c->nheads % c->ngroups != 0) return fail(REPLAY_ERR_SHAPE, "ngroups %d does not divide nheads %d", c->ngroups, c->nheads);
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0)
        return fail(REPLAY_ERR_SHAPE, "head_dim %d must be a multiple of 16 in [16, 256]", c->head_dim);
    const int R = c->state_dim;
    if (R != 16 && R != 32 && R != 64 && R != 128 && R != 256)
        return fail(REPLAY_ERR_SHAPE, "state_dim %d must be 16, 32, 64, 128 or 256", R);
    if (c->buf_cap < 1 || c->buf_cap > REPLAY_MAX_BUF)
        return fail(REPLAY_ERR_SHAPE, "buf_cap %d must be in [1, %d]", c->buf_cap, REPLAY_MAX_BUF);
    // the kernels split work item indices by multiplication (exact while index * divisor < 2^32)
    if ((long long)c->batch * c->nheads * (c->nheads > 256 ? c->nheads : 256) >= (1LL << 32))
        return fail(REPLAY_ERR_SHAPE, "batch * nheads * max(nheads, 256) must be below 2^32");
    if (c->io_dtype != REPLAY_F32 && c->io_dtype != REPLAY_BF16)
        return fail(REPLAY_ERR_DTYPE, "io_dtype must be REPLAY_F32 or REPLAY_BF16");
    if (c->ckpt_dtype != REPLAY_F32 && c->ckpt_dtype != REPLAY_F16 && c->ckpt_dtype != REPLAY_FP8_E4M3)
        return fail(REPLAY_ERR_DTYPE, "ckpt_dtype must be REPLAY_F32, REPLAY_F16 or REPLAY_FP8_E4M3");
    if (c->ckpt_dtype == REPLAY_FP8_E4M3 && c->read_copy == REPLAY_FP8_E4M3)
        return fail(REPLAY_ERR_UNSUPPORTED, "an FP8 checkpoint takes no FP8 read copy (it is one)");
    if (c->read_copy != REPLAY_NONE && c->read_copy != REPLAY_FP8_E4M3 && c->read_copy != REPLAY_MXFP4)
        return fail(REPLAY_ERR_DTYPE, "read_copy must be NONE, FP8_E4M3 or MXFP4");
    if (c->read_copy == REPLAY_MXFP4 && R % 32 != 0)
        return fail(REPLAY_ERR_SHAPE, "MXFP4 read copy needs state_dim divisible by 32");
    if (c->flags & ~(REPLAY_FLAG_VALU_FOLD | REPLAY_FLAG_QUANTIZED_CKPT | REPLAY_FLAG_STAGGER_FLUSH |
                     REPLAY_FLAG_MX_SCALE_CEIL))
        return fail(REPLAY_ERR_ARG, "unknown flags 0x%x", c->flags);
    if ((c->flags & REPLAY_FLAG_MX_SCALE_CEIL) && c->read_copy != REPLAY_MXFP4)
        return fail(REPLAY_ERR_ARG, "REPLAY_FLAG_MX_SCALE_CEIL applies to an MXFP4 read copy only");
    if ((c->flags & REPLAY_FLAG_QUANTIZED_CKPT) && c->read_copy == REPLAY_NONE)
        return fail(REPLAY_ERR_ARG, "REPLAY_FLAG_QUANTIZED_CKPT needs a read_copy format");
    if ((c->flags & REPLAY_FLAG_QUANTIZED_CKPT) && c->ckpt_dtype != REPLAY_F32)
        return fail(REPLAY_ERR_UNSUPPORTED, "REPLAY_FLAG_QUANTIZED_CKPT keeps an fp32 checkpoint");
    if ((c->flags & REPLAY_FLAG_VALU_FOLD) && (c->kind != REPLAY_MAMBA2 || c->ckpt_dtype != REPLAY_F32))
        return fail(REPLAY_ERR_UNSUPPORTED, "REPLAY_FLAG_VALU_FOLD is a Mamba-2 fp32-checkpoint cross-check");
    return ok();
}

void compute_layout(const replay_config* c, replay_layout* L)
{
    memset(L, 0, sizeof *L);
    const uint64_t B = c->batch, H = c->nheads, G = c->ngroups, C = c->head_dim, R = c->state_dim, cap = c->buf_cap;
    const uint64_t tiles = B * H, io = io_bytes(c);
    uint64_t off = 0;
    L->ckpt_off = off;
    L->ckpt_bytes = tiles * C * R * ckpt_bytes(c);
    off = align256(off + L->ckpt_bytes);
    if (c->read_copy == REPLAY_FP8_E4M3) L->rcopy_bytes = tiles * C * R;
    if (c->read_copy == REPLAY_MXFP4) {
        L->rcopy_bytes = tiles * C * R / 2;
        L->rscale_bytes = tiles * C * (R / 32);
    }
    L->rcopy_off = off;
    off = align256(off + L->rcopy_bytes);
    L->rscale_off = off;
    off = align256(off + L->rscale_bytes);
    L->buf_bytes[0] = 2 * B * H * cap * C * io;   // x (Mamba-2) / v (GDN)
    L->buf_bytes[1] = 2 * B * G * cap * R * io;   // B (Mamba-2) / k (GDN)
    L->buf_bytes[2] = 2 * B * H * cap * 4;        // dt (Mamba-2) / alpha (GDN), fp32
    L->buf_bytes[3] = c->kind == REPLAY_GDN ? 2 * B * H * cap * 4 : 0;  // beta
    for (int i = 0; i < 4; ++i) {
        L->buf_off[i] = off;
        off = align256(off + L->buf_bytes[i]);
    }
    L->book_off = off;
    L->book_bytes = 2 * 4 * B * 4;
    off = align256(off + L->book_bytes);
    L->err_off = off;
    off = align256(off + 4);
    L->total_bytes = off;
}

template <class T>
T* at(const replay_state* st, uint64_t off) { return reinterpret_cast<T*>(st->mem + off); }

int rc_kind(const replay_config* c)
{
    return c->read_copy == REPLAY_FP8_E4M3 ? rs::RC_FP8 : (c->read_copy == REPLAY_MXFP4 ? rs::RC_MXFP4 : rs::RC_NONE);
}

replay_status check_ptr(const void* p, const char* name)
{
    if (!p) return fail(REPLAY_ERR_ARG, "%s is NULL", name);
    if (!aligned(p, 16)) return fail(REPLAY_ERR_ALIGN, "%s is not 16-byte aligned", name);
    return REPLAY_OK;
}

// ---- paged key/value cache ----
bool page_size_ok(int32_t n) { return n == 16 || n == 32 || n == 64 || n == 128 || n == 256; }

int log2_of(int32_t n)
{
    int k = 0;
    while ((1 << k) < n) ++k;
    return k;
}

// Limits a table has to keep so that positions, units of work and page indices stay in 32 bits.
replay_status check_kv_table(int32_t batch, int32_t max_pages, int32_t page_size)
{
    if (batch < 1 || batch > 4096) return fail(REPLAY_ERR_SHAPE, "batch %d outside [1, 4096]", batch);
    if (max_pages < 1 || (long long)max_pages * page_size >= (1LL << 30) || (long long)batch * max_pages >= (1LL << 30))
        return fail(REPLAY_ERR_SHAPE, "max_pages %d: need >= 1, max_pages * page_size and batch * max_pages below 2^30",
                    max_pages);
    return REPLAY_OK;
}

replay_status check_kv_config(const replay_kv_config* c)
{
    if (!c) return fail(REPLAY_ERR_ARG, "kv config is NULL");
    if (c->abi_version != REPLAY_ABI_VERSION)
        return fail(REPLAY_ERR_ARG, "abi_version %d, library implements %d", c->abi_version, REPLAY_ABI_VERSION);
    if (!page_size_ok(c->page_size))
        return fail(REPLAY_ERR_SHAPE, "page_size %d must be 16, 32, 64, 128 or 256", c->page_size);
    if (c->npages < 1) return fail(REPLAY_ERR_SHAPE, "npages must be >= 1");
    return check_kv_table(c->batch, c->max_pages, c->page_size);
}

uint64_t kv_words(const replay_kv_config* c)
{
    const uint64_t bp = ((uint64_t)c->batch + 63) / 64 * 64;
    return 64 + 7 * bp + (uint64_t)c->batch * c->max_pages + (uint64_t)c->npages;
}

replay_status kv_pool(const replay_kv_config* c, void* mem, rs::KvPool* p)
{
    replay_status s = check_kv_config(c);
    if (s != REPLAY_OK) return s;
    if (!mem) return fail(REPLAY_ERR_ARG, "mem is NULL");
    if (!aligned(mem, 256)) return fail(REPLAY_ERR_ALIGN, "mem is not 256-byte aligned");
    const int bp = (c->batch + 63) / 64 * 64;
    int32_t* w = static_cast<int32_t*>(mem);
    *p = rs::KvPool{c->batch, c->npages, log2_of(c->page_size), c->max_pages, w, w + 64, w + 64 + bp, w + 64 + 2 * bp,
                    w + 64 + 3 * bp, w + 64 + 7 * bp, w + 64 + 7 * bp + (size_t)c->batch * c->max_pages, bp};
    return REPLAY_OK;
}

replay_status check_kv_layer(const replay_kv_layer* l)
{
    if (!l) return fail(REPLAY_ERR_ARG, "kv layer is NULL");
    if (l->abi_version != REPLAY_ABI_VERSION)
        return fail(REPLAY_ERR_ARG, "abi_version %d, library implements %d", l->abi_version, REPLAY_ABI_VERSION);
    if (l->io_dtype != REPLAY_BF16 && l->io_dtype != REPLAY_F16)
        return fail(REPLAY_ERR_DTYPE, "a paged cache's io_dtype must be REPLAY_BF16 or REPLAY_F16");
    if (l->cache_dtype != l->io_dtype && l->cache_dtype != REPLAY_FP8_E4M3)
        return fail(REPLAY_ERR_DTYPE, "cache_dtype must be io_dtype or REPLAY_FP8_E4M3");
    if (l->nkv < 1 || l->nheads < l->nkv || l->nheads % l->nkv != 0 || l->nheads > 4096)
        return fail(REPLAY_ERR_SHAPE, "nheads %d must be a multiple of nkv %d, at most 4096", l->nheads, l->nkv);
    if (l->head_dim != 64 && l->head_dim != 128 && l->head_dim != 256)
        return fail(REPLAY_ERR_UNSUPPORTED, "head dimension %d (64, 128 and 256 are built)", l->head_dim);
    if (!page_size_ok(l->page_size))
        return fail(REPLAY_ERR_SHAPE, "page_size %d must be 16, 32, 64, 128 or 256", l->page_size);
    if (l->npages < 1) return fail(REPLAY_ERR_SHAPE, "npages must be >= 1");
    if (l->rot_dim < 0 || l->rot_dim > l->head_dim || l->rot_dim % 16 != 0)
        return fail(REPLAY_ERR_SHAPE, "rot_dim %d must be a multiple of 16 in [0, head_dim]", l->rot_dim);
    if (l->rot_style != REPLAY_ROT_HALVES && l->rot_style != REPLAY_ROT_ADJACENT)
        return fail(REPLAY_ERR_ARG, "unknown rot_style %d", l->rot_style);
    return REPLAY_OK;
}

// Aligned as the elements of a small array are (per-sequence and per-row words may be slices).
replay_status check_words(const void* p, const char* name, uintptr_t size)
{
    if (!p) return fail(REPLAY_ERR_ARG, "%s is NULL", name);
    if (!aligned(p, size)) return fail(REPLAY_ERR_ALIGN, "%s is not %d-byte aligned", name, (int)size);
    return REPLAY_OK;
}

replay_status check_kv_scales(const replay_kv_layer* l, const float* k, const float* v)
{
    const bool fp8 = l->cache_dtype == REPLAY_FP8_E4M3;
    if (!fp8 && (k || v)) return fail(REPLAY_ERR_ARG, "k_scale and v_scale belong to an FP8 cache");
    replay_status s;
    if (fp8 && (s = check_words(k, "k_scale", 4)) != REPLAY_OK) return s;
    if (fp8 && (s = check_words(v, "v_scale", 4)) != REPLAY_OK) return s;
    return REPLAY_OK;
}

replay_status check_row_stride(int64_t stride, long long width, const char* name)
{
    if (stride < width || stride % 8 != 0 || stride >= (1LL << 31))
        return fail(REPLAY_ERR_ARG, "%s %lld must be >= %lld, a multiple of 8 and below 2^31", name, (long long)stride,
                    width);
    return REPLAY_OK;
}

uint64_t kv_meta_bytes(const rs::KvPlan& p) { return align256((uint64_t)p.nwg * 8); }
uint64_t kv_ml_bytes(const rs::KvPlan& p) { return align256((uint64_t)p.nwg * 2 * p.rpc * 8); }
uint64_t kv_ws_bytes(const rs::KvPlan& p, int D)
{
    return kv_meta_bytes(p) + kv_ml_bytes(p) + align256((uint64_t)p.nwg * 2 * p.rpc * D * 4);
}

// Sizes of an attention call, and how it is cut.
replay_status check_kv_call(const replay_kv_layer* l, int32_t batch, int32_t ntok, rs::KvPlan* plan)
{
    replay_status s = check_kv_layer(l);
    if (s != REPLAY_OK) return s;
    if (batch < 1 || batch > 4096) return fail(REPLAY_ERR_SHAPE, "batch %d outside [1, 4096]", batch);
    if (ntok < 1 || ntok > REPLAY_MAX_BUF) return fail(REPLAY_ERR_CAPACITY, "ntok = %d outside [1, %d]", ntok, REPLAY_MAX_BUF);
    *plan = rs::kv_attention_plan(l->head_dim, l->cache_dtype == REPLAY_FP8_E4M3, ntok * (l->nheads / l->nkv));
    return REPLAY_OK;
}

replay_status check_inputs(const replay_config* c, const replay_inputs* in, bool need_tokens, bool need_D)
{
    if (!in) return fail(REPLAY_ERR_ARG, "inputs are NULL");
    replay_status s;
    if (c->kind == REPLAY_MAMBA2) {
        if ((s = check_ptr(in->A, "A")) != REPLAY_OK) return s;
        if (need_D && (s = check_ptr(in->D, "D")) != REPLAY_OK) return s;
        if (need_tokens) {
            if ((s = check_ptr(in->x, "x")) != REPLAY_OK) return s;
            if ((s = check_ptr(in->B, "B")) != REPLAY_OK) return s;
            if ((s = check_ptr(in->C, "C")) != REPLAY_OK) return s;
            if ((s = check_ptr(in->dt, "dt")) != REPLAY_OK) return s;
        }
    } else if (need_tokens) {
        if ((s = check_ptr(in->q, "q")) != REPLAY_OK) return s;
        if ((s = check_ptr(in->k, "k")) != REPLAY_OK) return s;
        if ((s = check_ptr(in->v, "v")) != REPLAY_OK) return s;
        if ((s = check_ptr(in->alpha, "alpha")) != REPLAY_OK) return s;
        if ((s = check_ptr(in->beta, "beta")) != REPLAY_OK) return s;
    }
    return REPLAY_OK;
}

// Mamba-2 heads per workgroup: the heads of a group share the staged B and C rows
// and the sequence's bookkeeping, and a workgroup that serves several of them
// streams one head's checkpoint while it computes the previous head's outputs.
// Used with four waves per workgroup when the group size allows it.
// An fp32 or fp16 checkpoint without a read copy streams enough bytes per head
// that six single-head workgroups per SIMD hide the fixed work better (measured
// on the batch-256 layer: fp32 0.182 vs 0.192 ms per step, fp16 0.108 vs
// 0.110 ms); the lighter streams gain from the shared staging (FP8 checkpoint
// 0.091 -> 0.077 ms, read copies 0.10-0.29 -> 0.07-0.11 ms).
int mamba2_heads_per_wg(const replay_config* c, int wpg)
{
    if (c->kind != REPLAY_MAMBA2 || wpg != 4) return 1;
    if (c->ckpt_dtype != REPLAY_FP8_E4M3 && c->read_copy == REPLAY_NONE) return 1;
    return (c->nheads / c->ngroups) % 4 == 0 ? 4 : 1;
}

// Multipliers for div_magic / div_small (the kernels' divisions by launch-invariant
// divisors): floor(2^32 / d) + 1, exact for quotients of n with n d < 2^32 (0 for
// d = 1); and ceil(2^20 / d), exact for n < 2^20 / d.
uint32_t magic_div(uint32_t d)
{
    return d <= 1 ? 0u : (uint32_t)((1ull << 32) / d + 1);
}

int magic_div20(int d)
{
    return (int)(((1u << 20) + (uint32_t)d - 1) / (uint32_t)d);
}

// GDN strips per wave.  Every wave of a head runs the head's adjoint chain and
// stages its entries, so a wave that owns two strips halves that work per head.
// Used where the value rows of a head fill whole workgroups of four waves with
// two strips each (d_v a multiple of 128), d_k = 128, and the step streams
// fewer bytes than an fp32 checkpoint (an fp16 or FP8 checkpoint or a read
// copy): there the fixed work per head bounds the step.  An fp32 stream keeps
// one strip per wave: six waves per SIMD keep more loads in flight than four
// (measured on the batch-256, 32-head layer: FP8 checkpoint 0.063 -> 0.054 ms
// per step with two strips; fp32 0.100 -> 0.119 ms).
int gdn_strips_per_wave(const replay_config* c)
{
    if (c->kind != REPLAY_GDN || c->state_dim != 128 || c->head_dim % 128 != 0) return 1;
    return c->ckpt_dtype == REPLAY_F32 && c->read_copy == REPLAY_NONE ? 1 : 2;
}

rs::StepArgs step_args(const replay_state* st, const replay_inputs* in, void* y, int mode, int T,
                       const uint8_t* active)
{
    const replay_config* c = &st->cfg;
    rs::StepArgs a;
    memset(&a, 0, sizeof a);
    a.B = c->batch;
    a.H = c->nheads;
    a.G = c->ngroups;
    a.hpg = c->nheads / c->ngroups;
    a.C = c->head_dim;
    a.R = c->state_dim;
    a.cap = c->buf_cap;
    a.parity = st->parity;
    a.mode = mode;
    a.T = T;
    a.vmax = mode == rs::MODE_DECODE ? c->buf_cap + 1 : (mode == rs::MODE_FLUSH ? c->buf_cap : c->buf_cap + T);
    a.scale = c->scale;
    // workgroups of at most 4 waves, each wave owning spw 16-column strips: the
    // largest divisor of the wave count that is <= 4 sets the waves per workgroup
    const int strips = c->head_dim / 16;
    a.spw = gdn_strips_per_wave(c);
    int wpg = 1;
    for (int d = 4; d >= 1; --d)
        if ((strips / a.spw) % d == 0) { wpg = d; break; }
    a.nsplit = strips / a.spw / wpg;
    a.ht = mamba2_heads_per_wg(c, wpg);
    a.cw = c->head_dim / a.nsplit;
    a.mg_nsplit = magic_div((uint32_t)a.nsplit);
    a.mg_tiles = magic_div((uint32_t)(c->nheads / a.ht));
    a.mg_hpg = magic_div((uint32_t)a.hpg);
    a.m20_cx = magic_div20(a.cw / (c->io_dtype == REPLAY_BF16 ? 8 : 4));
    a.qckpt = (c->flags & REPLAY_FLAG_QUANTIZED_CKPT) ? 1 : 0;
    a.mxceil = (c->flags & REPLAY_FLAG_MX_SCALE_CEIL) ? 1 : 0;
    const replay_layout& L = st->lay;
    a.ckpt = at<void>(st, L.ckpt_off);
    a.rcopy = L.rcopy_bytes ? at<uint8_t>(st, L.rcopy_off) : nullptr;
    a.rscale = L.rscale_bytes ? at<uint8_t>(st, L.rscale_off) : nullptr;
    a.bufc = at<void>(st, L.buf_off[0]);
    a.bufr = at<void>(st, L.buf_off[1]);
    a.bufs0 = at<float>(st, L.buf_off[2]);
    a.bufs1 = L.buf_bytes[3] ? at<float>(st, L.buf_off[3]) : nullptr;
    const uint64_t B = c->batch, H = c->nheads, G = c->ngroups, cap = c->buf_cap;
    a.bank_c = B * H * cap * c->head_dim;
    a.bank_r = B * G * cap * c->state_dim;
    a.bank_s = B * H * cap;
    a.book = at<int32_t>(st, L.book_off);
    a.err = at<uint32_t>(st, L.err_off);
    if (st->stack) {                      // every member follows the stack's one bookkeeping set
        a.book = st->stack->book;
        a.err = st->stack->err;
        a.parity = st->stack->parity;
    }
    if (c->kind == REPLAY_MAMBA2) {
        a.in_c = in->x;
        a.in_r = in->B;
        a.in_q = in->C;
        a.in_s0 = in->dt;
        a.A = in->A;
        a.D = in->D;
    } else {
        a.in_c = in->v;
        a.in_r = in->k;
        a.in_q = in->q;
        a.in_s0 = in->alpha;
        a.in_s1 = in->beta;
    }
    a.y = y;
    a.active = active;
    return a;
}

replay_status launch_step(replay_state* st, const replay_inputs* in, void* y, int mode, int T, void* stream,
                          const uint8_t* active = nullptr)
{
    const replay_config* c = &st->cfg;
    rs::StepArgs a = step_args(st, in, y, mode, T, active);
    (void)fresh();
    const int io = c->io_dtype == REPLAY_BF16 ? rs::IO_BF16 : rs::IO_F32;
    const int rc = rc_kind(c);
    hipError_t e;
    const hipStream_t hs = (hipStream_t)stream;
    const int ck = ck_kind(c);
    if (c->kind == REPLAY_MAMBA2)
        e = ck == rs::CK_F16   ? rs::launch_mamba2_step_f16(a, io, rc, hs)
            : ck == rs::CK_FP8 ? rs::launch_mamba2_step_fp8(a, io, rc, hs)
                               : rs::launch_mamba2_step_f32(a, io, rc, (c->flags & REPLAY_FLAG_VALU_FOLD) != 0, hs);
    else
        e = ck == rs::CK_F16   ? rs::launch_gdn_step_f16(a, io, rc, hs)
            : ck == rs::CK_FP8 ? rs::launch_gdn_step_fp8(a, io, rc, hs)
                               : rs::launch_gdn_step_f32(a, io, rc, hs);
    replay_status s = hip_check(e, "replay step launch");
    if (s == REPLAY_OK && !st->stack) st->parity ^= 1;
    return s;
}

}  // namespace

extern "C" {

int32_t replay_abi_version(void) { return REPLAY_ABI_VERSION; }

const char* replay_status_str(int32_t s)
{
    switch (s) {
        case REPLAY_OK: return "ok";
        case REPLAY_ERR_ARG: return "invalid argument";
        case REPLAY_ERR_SHAPE: return "unsupported or inconsistent shape";
        case REPLAY_ERR_DTYPE: return "unsupported dtype";
        case REPLAY_ERR_ALIGN: return "misaligned pointer or short region";
        case REPLAY_ERR_STATE: return "operation not allowed in the current phase";
        case REPLAY_ERR_CAPACITY: return "draft count outside [1, buf_cap]";
        case REPLAY_ERR_UNSUPPORTED: return "not supported by this build";
        case REPLAY_ERR_HIP: return "HIP runtime error";
    }
    return "unknown status";
}

const char* replay_last_error(void) { return g_err.c_str(); }

replay_status replay_config_check(const replay_config* cfg) { return check_config(cfg); }

size_t replay_state_bytes(const replay_config* cfg)
{
    if (check_config(cfg) != REPLAY_OK) return 0;
    replay_layout L;
    compute_layout(cfg, &L);
    return (size_t)L.total_bytes;
}

replay_status replay_state_alloc(const replay_config* cfg, void* dev_mem, size_t bytes, void* stream,
                                 replay_state** out)
{
    replay_status s = check_config(cfg);
    if (s != REPLAY_OK) return s;
    if (!out) return fail(REPLAY_ERR_ARG, "out is NULL");
    if (!dev_mem) return fail(REPLAY_ERR_ARG, "dev_mem is NULL");
    if (!aligned(dev_mem, 256)) return fail(REPLAY_ERR_ALIGN, "state region must be 256-byte aligned");
    replay_layout L;
    compute_layout(cfg, &L);
    if (bytes < L.total_bytes)
        return fail(REPLAY_ERR_ALIGN, "state region has %zu bytes, needs %llu", bytes, (unsigned long long)L.total_bytes);
    replay_state* st = new replay_state;
    st->cfg = *cfg;
    st->mem = static_cast<uint8_t*>(dev_mem);
    st->bytes = bytes;
    st->lay = L;
    st->parity = 0;
    st->phase = 0;
    s = LAUNCH(rs::launch_fill_zero(dev_mem, L.total_bytes, (hipStream_t)stream), "state initialisation");
    if (s == REPLAY_OK)
        s = LAUNCH(rs::launch_book_reset(at<int32_t>(st, L.book_off), at<uint32_t>(st, L.err_off), cfg->batch, 0,
                                            cfg->buf_cap, (cfg->flags & REPLAY_FLAG_STAGGER_FLUSH) != 0,
                                            (hipStream_t)stream),
                      "bookkeeping initialisation");
    if (s != REPLAY_OK) {
        delete st;
        return s;
    }
    *out = st;
    return ok();
}

replay_status replay_state_free(replay_state* st)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is bound to a stack: free the stack first");
    delete st;
    return ok();
}

replay_status replay_state_layout(const replay_state* st, replay_layout* out)
{
    if (!st || !out) return fail(REPLAY_ERR_ARG, "NULL argument");
    *out = st->lay;
    return ok();
}

int32_t replay_state_phase(const replay_state* st) { return st ? st->phase : -1; }

static replay_status load_impl(replay_state* st, const void* S, bool src_f32, void* stream);

replay_status replay_load_checkpoint(replay_state* st, const void* S, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: load through the stack");
    if (st->phase != 0) return fail(REPLAY_ERR_STATE, "load while drafts are pending");
    replay_status s = load_impl(st, S, false, stream);
    if (s == REPLAY_OK) st->needs_load = false;
    return s;
}

replay_status replay_load_checkpoint_f32(replay_state* st, const float* S, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: load through the stack");
    if (st->phase != 0) return fail(REPLAY_ERR_STATE, "load while drafts are pending");
    replay_status s = load_impl(st, S, true, stream);
    if (s == REPLAY_OK) st->needs_load = false;
    return s;
}

// Checkpoint tiles and read copy of the tiles `m` names (all of them for a
// whole-state load), from `ntiles` source tiles.
static replay_status load_tiles(replay_state* st, const void* S, bool src_f32, int ntiles, const rs::SlotMap& m,
                                hipStream_t hs)
{
    const replay_config* c = &st->cfg;
    replay_status s = LAUNCH(rs::launch_logical_to_tiles(S, at<void>(st, st->lay.ckpt_off), ntiles, c->head_dim,
                                                         c->state_dim, ck_kind(c), src_f32, m, hs),
                             "checkpoint load");
    if (s != REPLAY_OK || c->read_copy == REPLAY_NONE) return s;
    return LAUNCH(rs::launch_quantize_read_copy(at<void>(st, st->lay.ckpt_off), at<uint8_t>(st, st->lay.rcopy_off),
                                                st->lay.rscale_bytes ? at<uint8_t>(st, st->lay.rscale_off) : nullptr,
                                                ntiles, c->head_dim, c->state_dim, rc_kind(c), ck_kind(c),
                                                (c->flags & REPLAY_FLAG_QUANTIZED_CKPT) != 0,
                                                (c->flags & REPLAY_FLAG_MX_SCALE_CEIL) != 0, m, hs),
                  "read copy quantize");
}

// Checkpoint tiles and read copy of one state, then its bookkeeping (the
// stack's, for a member).
static replay_status load_impl(replay_state* st, const void* S, bool src_f32, void* stream)
{
    replay_status s = check_ptr(S, "S_logical");
    if (s != REPLAY_OK) return s;
    const replay_config* c = &st->cfg;
    hipStream_t hs = (hipStream_t)stream;
    s = load_tiles(st, S, src_f32, c->batch * c->nheads, all_tiles(c->nheads), hs);
    if (s != REPLAY_OK || st->stack) return s;
    return LAUNCH(rs::launch_book_reset(at<int32_t>(st, st->lay.book_off), at<uint32_t>(st, st->lay.err_off),
                                        c->batch, st->parity, c->buf_cap,
                                        (c->flags & REPLAY_FLAG_STAGGER_FLUSH) != 0, hs),
                  "bookkeeping reset");
}

// Host-side checks of a per-slot load's sequence list: 1 <= n <= B, every slot
// in [0, B), no slot twice.
static replay_status check_slots(int32_t n, const int32_t* slots, int B)
{
    if (n < 1 || n > B) return fail(REPLAY_ERR_ARG, "slot count %d outside [1, %d]", n, B);
    if (!slots) return fail(REPLAY_ERR_ARG, "slots is NULL");
    std::vector<char> seen((size_t)B, 0);
    for (int32_t i = 0; i < n; ++i) {
        const int32_t b = slots[i];
        if (b < 0 || b >= B) return fail(REPLAY_ERR_ARG, "slot %d outside [0, %d)", b, B);
        if (seen[(size_t)b]) return fail(REPLAY_ERR_ARG, "slot %d listed twice", b);
        seen[(size_t)b] = 1;
    }
    return REPLAY_OK;
}

// The listed sequences' checkpoints (fp32 source [n][H][rows][cols]) and read
// copies, in chunks of SLOT_CHUNK sequences per launch; then, unless the state
// is a stack member, their bookkeeping.
static replay_status load_slots_impl(replay_state* st, int32_t n, const int32_t* slots, const float* S, hipStream_t hs)
{
    const replay_config* c = &st->cfg;
    const size_t seq_floats = (size_t)c->nheads * c->head_dim * c->state_dim;
    for (int32_t i0 = 0; i0 < n; i0 += rs::SLOT_CHUNK) {
        rs::SlotMap m;
        m.n = n - i0 < rs::SLOT_CHUNK ? n - i0 : rs::SLOT_CHUNK;
        m.H = c->nheads;
        for (int i = 0; i < m.n; ++i) m.slot[i] = slots[i0 + i];
        replay_status s = load_tiles(st, S + (size_t)i0 * seq_floats, true, m.n * c->nheads, m, hs);
        if (s != REPLAY_OK) return s;
        if (!st->stack) {
            s = LAUNCH(rs::launch_book_reset_slots(at<int32_t>(st, st->lay.book_off), c->batch, st->parity,
                                                   c->buf_cap, m, hs),
                       "slot bookkeeping reset");
            if (s != REPLAY_OK) return s;
        }
    }
    return REPLAY_OK;
}

replay_status replay_load_slots(replay_state* st, int32_t n, const int32_t* slots, const float* S, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: load through the stack");
    if (st->needs_load) return fail(REPLAY_ERR_STATE, "a former stack member must be loaded first");
    if (st->phase != 0) return fail(REPLAY_ERR_STATE, "load while drafts are pending");
    replay_status s = check_slots(n, slots, st->cfg.batch);
    if (s != REPLAY_OK) return s;
    if ((s = check_ptr(S, "S_logical")) != REPLAY_OK) return s;
    if ((s = load_slots_impl(st, n, slots, S, (hipStream_t)stream)) != REPLAY_OK) return s;
    return ok();
}

replay_status replay_read_checkpoint(const replay_state* st, void* out, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    replay_status s = check_ptr(out, "S_out");
    if (s != REPLAY_OK) return s;
    const replay_config* c = &st->cfg;
    return LAUNCH(rs::launch_tiles_to_logical(at<void>(st, st->lay.ckpt_off), out, c->batch * c->nheads,
                                                 c->head_dim, c->state_dim, ck_kind(c), (hipStream_t)stream),
                     "checkpoint read");
}

replay_status replay_read_copy(const replay_state* st, uint8_t* codes_out, uint8_t* scales_out, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    const replay_config* c = &st->cfg;
    if (c->read_copy == REPLAY_NONE) return fail(REPLAY_ERR_STATE, "state has no read copy");
    if (!codes_out) return fail(REPLAY_ERR_ARG, "codes_out is NULL");
    if (c->read_copy == REPLAY_MXFP4 && !scales_out) return fail(REPLAY_ERR_ARG, "scales_out is NULL");
    return LAUNCH(rs::launch_read_copy_to_logical(at<uint8_t>(st, st->lay.rcopy_off),
                                                     st->lay.rscale_bytes ? at<uint8_t>(st, st->lay.rscale_off) : nullptr,
                                                     codes_out, scales_out, c->batch * c->nheads, c->head_dim,
                                                     c->state_dim, rc_kind(c), (hipStream_t)stream),
                     "read copy export");
}

static replay_status read_book_impl(const int32_t* book, const uint32_t* err, int B, int parity, int32_t* book_out,
                                    uint32_t* err_out, void* stream)
{
    if (!book_out) return fail(REPLAY_ERR_ARG, "book_out is NULL");
    const size_t n = (size_t)3 * B * sizeof(int32_t);
    hipStream_t hs = (hipStream_t)stream;
    replay_status s = LAUNCH(hipMemcpyAsync(book_out, book + (size_t)parity * 4 * B, n, hipMemcpyDeviceToDevice, hs),
                                "bookkeeping copy");
    if (s != REPLAY_OK || !err_out) return s;
    return LAUNCH(hipMemcpyAsync(err_out, err, 4, hipMemcpyDeviceToDevice, hs), "error word copy");
}

replay_status replay_read_book(const replay_state* st, int32_t* book_out, uint32_t* err_out, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: read the stack's bookkeeping");
    return read_book_impl(at<int32_t>(st, st->lay.book_off), at<uint32_t>(st, st->lay.err_off), st->cfg.batch,
                          st->parity, book_out, err_out, stream);
}

static replay_status decode_impl(replay_state* st, const replay_inputs* in, const uint8_t* active, void* y,
                                 void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: step it through the stack");
    if (st->needs_load) return fail(REPLAY_ERR_STATE, "a former stack member must be loaded first");
    if (st->phase != 0) return fail(REPLAY_ERR_STATE, "decode while drafts are pending");
    replay_status s = check_inputs(&st->cfg, in, true, true);
    if (s != REPLAY_OK) return s;
    if ((s = check_ptr(y, "y")) != REPLAY_OK) return s;
    return launch_step(st, in, y, rs::MODE_DECODE, 1, stream, active);
}

replay_status replay_decode_step(replay_state* st, const replay_inputs* in, void* y, void* stream)
{
    return decode_impl(st, in, nullptr, y, stream);
}

replay_status replay_decode_step_masked(replay_state* st, const replay_inputs* in, const uint8_t* active, void* y,
                                        void* stream)
{
    if (!active) return fail(REPLAY_ERR_ARG, "active is NULL");
    return decode_impl(st, in, active, y, stream);
}

replay_status replay_flush(replay_state* st, const replay_inputs* in, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: step it through the stack");
    if (st->needs_load) return fail(REPLAY_ERR_STATE, "a former stack member must be loaded first");
    if (st->phase != 0) return fail(REPLAY_ERR_STATE, "flush while drafts are pending");
    replay_inputs none;
    memset(&none, 0, sizeof none);
    if (!in) in = &none;
    if (st->cfg.kind == REPLAY_MAMBA2) {
        replay_status s = check_ptr(in->A, "A");
        if (s != REPLAY_OK) return s;
    }
    return launch_step(st, in, nullptr, rs::MODE_FLUSH, 0, stream);
}

static replay_status spec_impl(replay_state* st, int32_t k, const replay_inputs* drafts, const uint8_t* active,
                               void* y, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: step it through the stack");
    if (st->needs_load) return fail(REPLAY_ERR_STATE, "a former stack member must be loaded first");
    if (st->phase != 0) return fail(REPLAY_ERR_STATE, "spec_append while drafts are pending");
    if (k < 1 || k > st->cfg.buf_cap) return fail(REPLAY_ERR_CAPACITY, "k = %d outside [1, %d]", k, st->cfg.buf_cap);
    replay_status s = check_inputs(&st->cfg, drafts, true, true);
    if (s != REPLAY_OK) return s;
    if ((s = check_ptr(y, "y")) != REPLAY_OK) return s;
    s = launch_step(st, drafts, y, rs::MODE_SPEC, k, stream, active);
    if (s == REPLAY_OK) st->phase = 1;
    return s;
}

replay_status replay_spec_append(replay_state* st, int32_t k, const replay_inputs* drafts, void* y, void* stream)
{
    return spec_impl(st, k, drafts, nullptr, y, stream);
}

replay_status replay_spec_append_masked(replay_state* st, int32_t k, const replay_inputs* drafts,
                                        const uint8_t* active, void* y, void* stream)
{
    if (!active) return fail(REPLAY_ERR_ARG, "active is NULL");
    return spec_impl(st, k, drafts, active, y, stream);
}

static replay_status commit_impl(replay_state* st, const int32_t* accepted, void* stream)
{
    if (st->phase != 1) return fail(REPLAY_ERR_STATE, "no drafts pending");
    replay_status s = LAUNCH(rs::launch_book_commit(at<int32_t>(st, st->lay.book_off), at<uint32_t>(st, st->lay.err_off),
                                                       st->cfg.batch, st->parity, accepted, (hipStream_t)stream),
                                "commit");
    if (s == REPLAY_OK) {
        st->parity ^= 1;
        st->phase = 0;
    }
    return s;
}

replay_status replay_spec_commit(replay_state* st, const int32_t* accepted, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: step it through the stack");
    if (st->needs_load) return fail(REPLAY_ERR_STATE, "a former stack member must be loaded first");
    if (!accepted) return fail(REPLAY_ERR_ARG, "accepted is NULL");
    if (!aligned(accepted, 4)) return fail(REPLAY_ERR_ALIGN, "accepted is not 4-byte aligned");
    return commit_impl(st, accepted, stream);
}

replay_status replay_spec_rollback(replay_state* st, void* stream)
{
    if (!st) return fail(REPLAY_ERR_ARG, "state is NULL");
    if (st->stack) return fail(REPLAY_ERR_STATE, "the state is a stack member: step it through the stack");
    if (st->needs_load) return fail(REPLAY_ERR_STATE, "a former stack member must be loaded first");
    return commit_impl(st, nullptr, stream);
}

// ---- layer stacks: one bookkeeping set for every SSM layer of a model --------

static replay_status stack_check_step(const replay_stack* stk, int32_t layer, int mode, int k, const uint8_t* active)
{
    if (!stk) return fail(REPLAY_ERR_ARG, "stack is NULL");
    const int n = (int)stk->layers.size();
    if (layer < 0 || layer >= n) return fail(REPLAY_ERR_ARG, "layer %d outside [0, %d)", layer, n);
    if (layer != stk->next)
        return fail(REPLAY_ERR_STATE, "layer %d stepped out of order: the step expects layer %d", layer, stk->next);
    if (stk->next == 0 && stk->phase != 0) return fail(REPLAY_ERR_STATE, "drafts are pending");
    if (stk->next > 0 && (mode != stk->step_mode || k != stk->step_k))
        return fail(REPLAY_ERR_STATE, "every layer of a step runs the same operation with the same draft count");
    if (stk->next > 0 && active != stk->step_active)
        return fail(REPLAY_ERR_STATE, "every layer of a step uses the same active mask");
    return REPLAY_OK;
}

// A layer of the step ran: after the last one the shared bookkeeping copy
// written by the step becomes the current one.
static void stack_advance(replay_stack* stk, int mode, int k, const uint8_t* active)
{
    if (stk->next == 0) {
        stk->step_mode = mode;
        stk->step_k = k;
        stk->step_active = active;
    }
    if (++stk->next == (int)stk->layers.size()) {
        stk->next = 0;
        stk->parity ^= 1;
        stk->step_mode = -1;
        if (mode == rs::MODE_SPEC) stk->phase = 1;
    }
}

static replay_status stack_idle(const replay_stack* stk, const char* what)
{
    if (!stk) return fail(REPLAY_ERR_ARG, "stack is NULL");
    if (stk->next != 0) return fail(REPLAY_ERR_STATE, "%s in the middle of a step (layer %d is next)", what, stk->next);
    return REPLAY_OK;
}

static replay_status stack_reset_book(replay_stack* stk, void* stream)
{
    const replay_config* c = &stk->layers[0]->cfg;
    return LAUNCH(rs::launch_book_reset(stk->book, stk->err, c->batch, stk->parity, c->buf_cap,
                                           (c->flags & REPLAY_FLAG_STAGGER_FLUSH) != 0, (hipStream_t)stream),
                     "bookkeeping reset");
}

replay_status replay_stack_create(replay_state* const* layers, int32_t nlayers, void* stream, replay_stack** out)
{
    if (!out) return fail(REPLAY_ERR_ARG, "out is NULL");
    if (!layers || nlayers < 1) return fail(REPLAY_ERR_ARG, "a stack needs at least one layer");
    const replay_config* c0 = layers[0] ? &layers[0]->cfg : nullptr;
    for (int l = 0; l < nlayers; ++l) {
        const replay_state* st = layers[l];
        if (!st) return fail(REPLAY_ERR_ARG, "layer %d is NULL", l);
        for (int m = 0; m < l; ++m)
            if (layers[m] == st) return fail(REPLAY_ERR_ARG, "layer %d repeats layer %d", l, m);
        if (st->stack) return fail(REPLAY_ERR_STATE, "layer %d already belongs to a stack", l);
        if (st->phase != 0) return fail(REPLAY_ERR_STATE, "layer %d has pending drafts", l);
        const replay_config* c = &st->cfg;
        if (c->batch != c0->batch || c->buf_cap != c0->buf_cap)
            return fail(REPLAY_ERR_SHAPE, "layer %d: batch and buf_cap must match layer 0", l);
        if ((c->flags & REPLAY_FLAG_STAGGER_FLUSH) != (c0->flags & REPLAY_FLAG_STAGGER_FLUSH))
            return fail(REPLAY_ERR_ARG, "layer %d: REPLAY_FLAG_STAGGER_FLUSH must match layer 0", l);
    }
    replay_stack* stk = new replay_stack;
    stk->layers.assign(layers, layers + nlayers);
    stk->book = at<int32_t>(layers[0], layers[0]->lay.book_off);
    stk->err = at<uint32_t>(layers[0], layers[0]->lay.err_off);
    replay_status s = stack_reset_book(stk, stream);
    if (s != REPLAY_OK) {
        delete stk;
        return s;
    }
    for (replay_state* st : stk->layers) st->stack = stk;
    *out = stk;
    return ok();
}

replay_status replay_stack_free(replay_stack* stk)
{
    if (!stk) return fail(REPLAY_ERR_ARG, "stack is NULL");
    for (replay_state* st : stk->layers) {
        st->stack = nullptr;
        st->needs_load = true;
        st->phase = 0;
    }
    delete stk;
    return ok();
}

static replay_status stack_load_impl(replay_stack* stk, const void* const* S, bool src_f32, void* stream)
{
    replay_status s = stack_idle(stk, "load");
    if (s != REPLAY_OK) return s;
    if (stk->phase != 0) return fail(REPLAY_ERR_STATE, "load while drafts are pending");
    if (!S) return fail(REPLAY_ERR_ARG, "S_logical is NULL");
    for (size_t l = 0; l < stk->layers.size(); ++l)
        if ((s = check_ptr(S[l], "S_logical[layer]")) != REPLAY_OK) return s;
    for (size_t l = 0; l < stk->layers.size(); ++l)
        if ((s = load_impl(stk->layers[l], S[l], src_f32, stream)) != REPLAY_OK) return s;
    return stack_reset_book(stk, stream);
}

replay_status replay_stack_load(replay_stack* stk, const void* const* S, void* stream)
{
    return stack_load_impl(stk, S, false, stream);
}

replay_status replay_stack_load_f32(replay_stack* stk, const float* const* S, void* stream)
{
    return stack_load_impl(stk, reinterpret_cast<const void* const*>(S), true, stream);
}

replay_status replay_stack_load_slots(replay_stack* stk, int32_t n, const int32_t* slots, const float* const* S,
                                      void* stream)
{
    replay_status s = stack_idle(stk, "load");
    if (s != REPLAY_OK) return s;
    if (stk->phase != 0) return fail(REPLAY_ERR_STATE, "load while drafts are pending");
    const replay_config* c0 = &stk->layers[0]->cfg;
    if ((s = check_slots(n, slots, c0->batch)) != REPLAY_OK) return s;
    if (!S) return fail(REPLAY_ERR_ARG, "S_logical is NULL");
    for (size_t l = 0; l < stk->layers.size(); ++l)
        if ((s = check_ptr(S[l], "S_logical[layer]")) != REPLAY_OK) return s;
    hipStream_t hs = (hipStream_t)stream;
    for (size_t l = 0; l < stk->layers.size(); ++l)
        if ((s = load_slots_impl(stk->layers[l], n, slots, S[l], hs)) != REPLAY_OK) return s;
    for (int32_t i0 = 0; i0 < n; i0 += rs::SLOT_CHUNK) {
        rs::SlotMap m;
        m.n = n - i0 < rs::SLOT_CHUNK ? n - i0 : rs::SLOT_CHUNK;
        m.H = 1;
        for (int i = 0; i < m.n; ++i) m.slot[i] = slots[i0 + i];
        s = LAUNCH(rs::launch_book_reset_slots(stk->book, c0->batch, stk->parity, c0->buf_cap, m, hs),
                   "slot bookkeeping reset");
        if (s != REPLAY_OK) return s;
    }
    return ok();
}

static replay_status stack_decode_impl(replay_stack* stk, int32_t layer, const replay_inputs* in,
                                       const uint8_t* active, void* y, void* stream)
{
    replay_status s = stack_check_step(stk, layer, rs::MODE_DECODE, 1, active);
    if (s != REPLAY_OK) return s;
    replay_state* st = stk->layers[layer];
    if ((s = check_inputs(&st->cfg, in, true, true)) != REPLAY_OK) return s;
    if ((s = check_ptr(y, "y")) != REPLAY_OK) return s;
    if ((s = launch_step(st, in, y, rs::MODE_DECODE, 1, stream, active)) != REPLAY_OK) return s;
    stack_advance(stk, rs::MODE_DECODE, 1, active);
    return ok();
}

replay_status replay_stack_decode_layer(replay_stack* stk, int32_t layer, const replay_inputs* in, void* y,
                                        void* stream)
{
    return stack_decode_impl(stk, layer, in, nullptr, y, stream);
}

replay_status replay_stack_decode_layer_masked(replay_stack* stk, int32_t layer, const replay_inputs* in,
                                               const uint8_t* active, void* y, void* stream)
{
    if (!active) return fail(REPLAY_ERR_ARG, "active is NULL");
    return stack_decode_impl(stk, layer, in, active, y, stream);
}

static replay_status stack_spec_impl(replay_stack* stk, int32_t layer, int32_t k, const replay_inputs* drafts,
                                     const uint8_t* active, void* y, void* stream)
{
    replay_status s = stack_check_step(stk, layer, rs::MODE_SPEC, k, active);
    if (s != REPLAY_OK) return s;
    replay_state* st = stk->layers[layer];
    if (k < 1 || k > st->cfg.buf_cap) return fail(REPLAY_ERR_CAPACITY, "k = %d outside [1, %d]", k, st->cfg.buf_cap);
    if ((s = check_inputs(&st->cfg, drafts, true, true)) != REPLAY_OK) return s;
    if ((s = check_ptr(y, "y")) != REPLAY_OK) return s;
    if ((s = launch_step(st, drafts, y, rs::MODE_SPEC, k, stream, active)) != REPLAY_OK) return s;
    stack_advance(stk, rs::MODE_SPEC, k, active);
    return ok();
}

replay_status replay_stack_spec_layer(replay_stack* stk, int32_t layer, int32_t k, const replay_inputs* drafts,
                                      void* y, void* stream)
{
    return stack_spec_impl(stk, layer, k, drafts, nullptr, y, stream);
}

replay_status replay_stack_spec_layer_masked(replay_stack* stk, int32_t layer, int32_t k, const replay_inputs* drafts,
                                             const uint8_t* active, void* y, void* stream)
{
    if (!active) return fail(REPLAY_ERR_ARG, "active is NULL");
    return stack_spec_impl(stk, layer, k, drafts, active, y, stream);
}

replay_status replay_stack_flush(replay_stack* stk, const replay_inputs* const* in, void* stream)
{
    replay_status s = stack_idle(stk, "flush");
    if (s != REPLAY_OK) return s;
    if (stk->phase != 0) return fail(REPLAY_ERR_STATE, "flush while drafts are pending");
    replay_inputs none;
    memset(&none, 0, sizeof none);
    for (size_t l = 0; l < stk->layers.size(); ++l) {
        const replay_inputs* il = (in && in[l]) ? in[l] : &none;
        if (stk->layers[l]->cfg.kind == REPLAY_MAMBA2 && (s = check_ptr(il->A, "A")) != REPLAY_OK) return s;
    }
    for (size_t l = 0; l < stk->layers.size(); ++l) {
        const replay_inputs* il = (in && in[l]) ? in[l] : &none;
        if ((s = launch_step(stk->layers[l], il, nullptr, rs::MODE_FLUSH, 0, stream)) != REPLAY_OK) return s;
    }
    stk->parity ^= 1;
    return ok();
}

static replay_status stack_commit_impl(replay_stack* stk, const int32_t* accepted, void* stream)
{
    replay_status s = stack_idle(stk, "commit");
    if (s != REPLAY_OK) return s;
    if (stk->phase != 1) return fail(REPLAY_ERR_STATE, "no drafts pending");
    s = LAUNCH(rs::launch_book_commit(stk->book, stk->err, stk->layers[0]->cfg.batch, stk->parity, accepted,
                                         (hipStream_t)stream),
                  "commit");
    if (s == REPLAY_OK) {
        stk->parity ^= 1;
        stk->phase = 0;
    }
    return s;
}

replay_status replay_stack_commit(replay_stack* stk, const int32_t* accepted, void* stream)
{
    if (!accepted) return fail(REPLAY_ERR_ARG, "accepted is NULL");
    if (!aligned(accepted, 4)) return fail(REPLAY_ERR_ALIGN, "accepted is not 4-byte aligned");
    return stack_commit_impl(stk, accepted, stream);
}

replay_status replay_stack_rollback(replay_stack* stk, void* stream) { return stack_commit_impl(stk, nullptr, stream); }

replay_status replay_stack_read_book(const replay_stack* stk, int32_t* book_out, uint32_t* err_out, void* stream)
{
    if (!stk) return fail(REPLAY_ERR_ARG, "stack is NULL");
    return read_book_impl(stk->book, stk->err, stk->layers[0]->cfg.batch, stk->parity, book_out, err_out, stream);
}

int32_t replay_stack_layers(const replay_stack* stk) { return stk ? (int32_t)stk->layers.size() : -1; }
int32_t replay_stack_next_layer(const replay_stack* stk) { return stk ? stk->next : -1; }
int32_t replay_stack_phase(const replay_stack* stk) { return stk ? stk->phase : -1; }

static replay_status conv_common(const replay_config* cfg, rs::ConvArgs* a, const replay_inputs* in, void* y, int T)
{
    replay_config c = *cfg;
    // the baselines have no checkpoint/buffer: read-copy, flag and kind limits
    // of the replay kernels do not apply
    c.read_copy = REPLAY_NONE;
    c.flags = 0;
    const int kind = c.kind;
    c.kind = REPLAY_MAMBA2;
    replay_status s = check_config(&c);
    if (s != REPLAY_OK) return s;
    c.kind = kind;
    if ((s = check_inputs(&c, in, true, true)) != REPLAY_OK) return s;
    if ((s = check_ptr(y, "y")) != REPLAY_OK) return s;
    memset(a, 0, sizeof *a);
    a->kind = kind == REPLAY_GDN ? 1 : 0;
    a->B = c.batch;
    a->H = c.nheads;
    a->G = c.ngroups;
    a->hpg = c.nheads / c.ngroups;
    a->C = c.head_dim;
    a->R = c.state_dim;
    a->T = T;
    a->scale = c.scale;
    if (kind == REPLAY_MAMBA2) {
        a->in_c = in->x;
        a->in_r = in->B;
        a->in_q = in->C;
        a->in_s0 = in->dt;
        a->A = in->A;
        a->D = in->D;
    } else {
        a->in_c = in->v;
        a->in_r = in->k;
        a->in_q = in->q;
        a->in_s0 = in->alpha;
        a->in_s1 = in->beta;
    }
    a->y = y;
    return REPLAY_OK;
}

replay_status replay_conv_decode_step(const replay_config* cfg, void* S, const replay_inputs* in, void* y,
                                      void* stream)
{
    rs::ConvArgs a;
    replay_status s = conv_common(cfg, &a, in, y, 1);
    if (s != REPLAY_OK) return s;
    if ((s = check_ptr(S, "S")) != REPLAY_OK) return s;
    a.S = S;
    return LAUNCH(rs::launch_conv_step(a, cfg->io_dtype == REPLAY_BF16 ? rs::IO_BF16 : rs::IO_F32, ck_kind(cfg),
                                          (hipStream_t)stream),
                     "conventional decode");
}

replay_status replay_conv_spec_step(const replay_config* cfg, const void* S, void* snaps, int32_t k,
                                    const replay_inputs* drafts, void* y, void* stream)
{
    rs::ConvArgs a;
    replay_status s = conv_common(cfg, &a, drafts, y, k);
    if (s != REPLAY_OK) return s;
    if (k < 1 || k > REPLAY_MAX_BUF) return fail(REPLAY_ERR_CAPACITY, "k = %d outside [1, %d]", k, REPLAY_MAX_BUF);
    if ((s = check_ptr(S, "S")) != REPLAY_OK) return s;
    if ((s = check_ptr(snaps, "snaps")) != REPLAY_OK) return s;
    a.S_in = S;
    a.S = const_cast<void*>(S);
    a.snaps = snaps;
    return LAUNCH(rs::launch_conv_step(a, cfg->io_dtype == REPLAY_BF16 ? rs::IO_BF16 : rs::IO_F32, ck_kind(cfg),
                                          (hipStream_t)stream),
                     "conventional spec step");
}

replay_status replay_conv_spec_restore(const replay_config* cfg, void* S, const void* snaps, int32_t k,
                                       const int32_t* accepted, void* stream)
{
    if (!cfg) return fail(REPLAY_ERR_ARG, "config is NULL");
    replay_status s;
    if ((s = check_ptr(S, "S")) != REPLAY_OK) return s;
    if ((s = check_ptr(snaps, "snaps")) != REPLAY_OK) return s;
    if (!accepted) return fail(REPLAY_ERR_ARG, "accepted is NULL");
    if (k < 1 || k > REPLAY_MAX_BUF) return fail(REPLAY_ERR_CAPACITY, "k = %d outside [1, %d]", k, REPLAY_MAX_BUF);
    replay_config c = *cfg;
    c.kind = REPLAY_MAMBA2;
    c.read_copy = REPLAY_NONE;
    c.flags = 0;
    if ((s = check_config(&c)) != REPLAY_OK) return s;
    const size_t tile_bytes = (size_t)cfg->head_dim * cfg->state_dim * ckpt_bytes(cfg);
    return LAUNCH(rs::launch_conv_restore(S, snaps, accepted, cfg->batch, tile_bytes, cfg->nheads, k,
                                             (hipStream_t)stream),
                     "conventional restore");
}

replay_status replay_standin_linear(const void* X, const void* W, void* Y, int32_t M, int32_t K, int32_t N,
                                    void* stream)
{
    replay_status s;
    if ((s = check_ptr(X, "X")) != REPLAY_OK) return s;
    if ((s = check_ptr(W, "W")) != REPLAY_OK) return s;
    if ((s = check_ptr(Y, "Y")) != REPLAY_OK) return s;
    if (M < 1 || K < 64 || K % 64 != 0 || N < 1)
        return fail(REPLAY_ERR_SHAPE, "linear needs M >= 1, K a positive multiple of 64 and N >= 1 (M %d, K %d, N %d)",
                    M, K, N);
    if ((long long)(M + 63) / 64 > 65535) return fail(REPLAY_ERR_SHAPE, "M %d too large", M);
    return LAUNCH(rs::launch_standin_linear(X, W, Y, M, K, N, (hipStream_t)stream), "stand-in linear");
}

replay_status replay_standin_attention(const void* q, int64_t q_stride, const void* K, const void* V, void* o,
                                       int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t L, float scale,
                                       void* stream)
{
    replay_status s;
    if ((s = check_ptr(q, "q")) != REPLAY_OK) return s;
    if ((s = check_ptr(K, "K")) != REPLAY_OK) return s;
    if ((s = check_ptr(V, "V")) != REPLAY_OK) return s;
    if ((s = check_ptr(o, "o")) != REPLAY_OK) return s;
    if (B < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || L < 1)
        return fail(REPLAY_ERR_SHAPE, "attention needs B, Hkv, L >= 1 and Hkv dividing Hq");
    const int qpk = Hq / Hkv;
    if (qpk != 1 && qpk != 2 && qpk != 4 && qpk != 8)
        return fail(REPLAY_ERR_UNSUPPORTED, "query heads per key/value head must be 1, 2, 4 or 8 (is %d)", qpk);
    if (D != 128) return fail(REPLAY_ERR_UNSUPPORTED, "head dimension %d (128 is built)", D);
    if (q_stride < (int64_t)Hq * D || q_stride % 8 != 0)
        return fail(REPLAY_ERR_ARG, "q_stride %lld must be >= Hq * D and a multiple of 8", (long long)q_stride);
    if ((long long)B * Hkv > (1LL << 31) - 1) return fail(REPLAY_ERR_SHAPE, "B * Hkv too large");
    return LAUNCH(rs::launch_standin_attention(q, K, V, o, B, Hq, Hkv, D, L, (size_t)q_stride, scale,
                                               (hipStream_t)stream),
                  "stand-in attention");
}

// ---- paged key/value cache ---------------------------------------------------
size_t replay_kv_bytes(const replay_kv_config* cfg)
{
    if (check_kv_config(cfg) != REPLAY_OK) return 0;
    (void)ok();
    return (size_t)(kv_words(cfg) * 4);
}

replay_status replay_kv_reset(const replay_kv_config* cfg, void* mem, void* stream)
{
    rs::KvPool p;
    const replay_status s = kv_pool(cfg, mem, &p);
    if (s != REPLAY_OK) return s;
    return LAUNCH(rs::launch_kv_reset(p, (hipStream_t)stream), "page pool reset");
}

replay_status replay_kv_reserve(const replay_kv_config* cfg, void* mem, int32_t ntok, const int32_t* counts,
                                const uint8_t* active, int32_t rows, int64_t* slots, int32_t* pos, int32_t* starts,
                                void* stream)
{
    rs::KvPool p;
    replay_status s = kv_pool(cfg, mem, &p);
    if (s != REPLAY_OK) return s;
    if ((s = check_words(slots, "slots", 8)) != REPLAY_OK) return s;
    if ((s = check_words(pos, "pos", 4)) != REPLAY_OK) return s;
    if (counts) {
        if ((s = check_words(counts, "counts", 4)) != REPLAY_OK) return s;
        if ((s = check_words(starts, "starts", 4)) != REPLAY_OK) return s;
        if (ntok != 0) return fail(REPLAY_ERR_ARG, "ntok must be 0 with counts");
        if (rows < 1) return fail(REPLAY_ERR_SHAPE, "rows must be >= 1");
    } else {
        if (starts) return fail(REPLAY_ERR_ARG, "starts belongs to counts");
        if (ntok < 1 || ntok > REPLAY_MAX_BUF)
            return fail(REPLAY_ERR_CAPACITY, "ntok = %d outside [1, %d]", ntok, REPLAY_MAX_BUF);
        if (rows < ntok * cfg->batch) return fail(REPLAY_ERR_SHAPE, "rows %d below ntok * batch", rows);
    }
    return LAUNCH(rs::launch_kv_reserve(p, ntok, counts, active, rows, slots, pos, starts, (hipStream_t)stream),
                  "page reserve");
}

replay_status replay_kv_commit(const replay_kv_config* cfg, void* mem, const int32_t* accepted, void* stream)
{
    rs::KvPool p;
    replay_status s = kv_pool(cfg, mem, &p);
    if (s != REPLAY_OK) return s;
    if (accepted && (s = check_words(accepted, "accepted", 4)) != REPLAY_OK) return s;
    return LAUNCH(rs::launch_kv_commit(p, accepted, (hipStream_t)stream), "page commit");
}

replay_status replay_kv_release(const replay_kv_config* cfg, void* mem, const uint8_t* mask, void* stream)
{
    rs::KvPool p;
    const replay_status s = kv_pool(cfg, mem, &p);
    if (s != REPLAY_OK) return s;
    return LAUNCH(rs::launch_kv_release(p, mask, (hipStream_t)stream), "page release");
}

replay_status replay_kv_append(const replay_kv_layer* layer, const replay_kv_append_args* args, void* stream)
{
    replay_status s = check_kv_layer(layer);
    if (s != REPLAY_OK) return s;
    if (!args) return fail(REPLAY_ERR_ARG, "append arguments are NULL");
    const replay_kv_append_args& x = *args;
    const int Hq = layer->nheads, Hkv = layer->nkv, D = layer->head_dim;
    // (two rows a workgroup of 256 lanes, and a launch holds less than 2^32 of them)
    if (x.rows < 0 || x.rows > (1 << 25) - 2) return fail(REPLAY_ERR_SHAPE, "rows %d outside [0, 2^25 - 2]", x.rows);
    if ((s = check_ptr(x.K, "K")) != REPLAY_OK) return s;
    if ((s = check_ptr(x.V, "V")) != REPLAY_OK) return s;
    if ((s = check_kv_scales(layer, x.k_scale, x.v_scale)) != REPLAY_OK) return s;
    if (!x.q != !x.q_out) return fail(REPLAY_ERR_ARG, "q and q_out go together");
    if (x.err && !aligned(x.err, 4)) return fail(REPLAY_ERR_ALIGN, "err is not 4-byte aligned");
    if (x.rows == 0) return ok();
    if ((s = check_ptr(x.k, "k")) != REPLAY_OK) return s;
    if ((s = check_ptr(x.v, "v")) != REPLAY_OK) return s;
    if ((s = check_row_stride(x.k_stride, (long long)Hkv * D, "k_stride")) != REPLAY_OK) return s;
    if ((s = check_row_stride(x.v_stride, (long long)Hkv * D, "v_stride")) != REPLAY_OK) return s;
    if (x.q) {
        if ((s = check_ptr(x.q, "q")) != REPLAY_OK) return s;
        if ((s = check_ptr(x.q_out, "q_out")) != REPLAY_OK) return s;
        if ((s = check_row_stride(x.q_stride, (long long)Hq * D, "q_stride")) != REPLAY_OK) return s;
    }
    if ((s = check_words(x.slots, "slots", 8)) != REPLAY_OK) return s;
    if (layer->rot_dim > 0) {
        if ((s = check_words(x.pos, "pos", 4)) != REPLAY_OK) return s;
        if ((s = check_words(x.freq, "freq", 4)) != REPLAY_OK) return s;
        if (x.naxes < 1 || x.naxes > 8) return fail(REPLAY_ERR_SHAPE, "naxes %d outside [1, 8]", x.naxes);
    }
    const rs::KvAppend a{x.q, x.k, x.v, x.q_stride, x.k_stride, x.v_stride, x.slots, x.pos, x.freq, x.axis, x.q_out,
                         x.K, x.V, x.k_scale, x.v_scale, x.err, x.naxes, x.rows, Hq, Hkv, D, log2_of(layer->page_size),
                         layer->rot_dim, (int64_t)layer->npages * layer->page_size};
    return LAUNCH(rs::launch_kv_append(a, layer->io_dtype == REPLAY_BF16 ? rs::KV_BF16 : rs::KV_F16,
                                       layer->cache_dtype == REPLAY_FP8_E4M3, layer->rot_style, (hipStream_t)stream),
                  "cache append");
}

size_t replay_kv_attention_workspace(const replay_kv_layer* layer, int32_t batch, int32_t ntok)
{
    rs::KvPlan p;
    if (check_kv_call(layer, batch, ntok, &p) != REPLAY_OK) return 0;
    (void)ok();
    return (size_t)kv_ws_bytes(p, layer->head_dim);
}

replay_status replay_kv_attention(const replay_kv_layer* layer, const replay_kv_attention_args* args, void* ws,
                                  size_t ws_bytes, void* stream)
{
    if (!args) return fail(REPLAY_ERR_ARG, "attention arguments are NULL");
    const replay_kv_attention_args& x = *args;
    rs::KvPlan p;
    replay_status s = check_kv_call(layer, x.batch, x.ntok, &p);
    if (s != REPLAY_OK) return s;
    const int Hq = layer->nheads, Hkv = layer->nkv, D = layer->head_dim;
    const bool fp8 = layer->cache_dtype == REPLAY_FP8_E4M3;
    if ((s = check_kv_table(x.batch, x.max_pages, layer->page_size)) != REPLAY_OK) return s;
    if ((s = check_ptr(x.q, "q")) != REPLAY_OK) return s;
    if ((s = check_row_stride(x.q_stride, (long long)Hq * D, "q_stride")) != REPLAY_OK) return s;
    if ((s = check_ptr(x.K, "K")) != REPLAY_OK) return s;
    if ((s = check_ptr(x.V, "V")) != REPLAY_OK) return s;
    if ((s = check_ptr(x.o, "o")) != REPLAY_OK) return s;
    if ((s = check_kv_scales(layer, x.k_scale, x.v_scale)) != REPLAY_OK) return s;
    if ((s = check_words(x.table, "table", 4)) != REPLAY_OK) return s;
    if ((s = check_words(x.end, "end", 4)) != REPLAY_OK) return s;
    if (x.lse && !aligned(x.lse, 4)) return fail(REPLAY_ERR_ALIGN, "lse is not 4-byte aligned");
    if (x.err && !aligned(x.err, 4)) return fail(REPLAY_ERR_ALIGN, "err is not 4-byte aligned");
    if (x.window < 0) return fail(REPLAY_ERR_ARG, "window %d is negative", x.window);
    if ((long long)x.batch * Hkv * p.nchunk * (((long long)x.max_pages * layer->page_size + 127) / 128 + 1) >= (1LL << 31))
        return fail(REPLAY_ERR_SHAPE, "batch * nkv * max_pages * page_size too large");
    if (!ws) return fail(REPLAY_ERR_ARG, "workspace is NULL");
    if (!aligned(ws, 256) || ws_bytes < kv_ws_bytes(p, D))
        return fail(REPLAY_ERR_ALIGN, "workspace needs %llu bytes, 256-byte aligned", (unsigned long long)kv_ws_bytes(p, D));
    uint8_t* w = static_cast<uint8_t*>(ws);
    rs::KvAttention a;
    a.q = x.q;
    a.q_stride = x.q_stride;
    a.K = x.K;
    a.V = x.V;
    a.k_scale = x.k_scale;
    a.v_scale = x.v_scale;
    a.table = x.table;
    a.end = x.end;
    a.active = x.active;
    a.o = x.o;
    a.lse = x.lse;
    a.err = x.err;
    a.meta = reinterpret_cast<int32_t*>(w);
    a.part_ml = reinterpret_cast<float*>(w + kv_meta_bytes(p));
    a.part_o = reinterpret_cast<float*>(w + kv_meta_bytes(p) + kv_ml_bytes(p));
    a.B = x.batch;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = Hq / Hkv;
    a.T = x.ntok;
    a.npages = layer->npages;
    a.page_shift = log2_of(layer->page_size);
    a.max_pages = x.max_pages;
    // a window past every position is none
    a.window = x.window < x.max_pages * layer->page_size ? x.window : 0;
    a.rows = x.ntok * a.group;
    a.rpc = p.rpc;
    a.nchunk = p.nchunk;
    // the most tokens a sequence's rows can see, in blocks of 32
    const long long cap = (long long)x.max_pages * layer->page_size, seen = (long long)a.window + x.ntok - 1 + 31;
    // (short ranges are over sooner than their order is found: 2048 of 200 tokens 47 us as they stand, 58 by length)
    const long long most = a.window > 0 && seen < cap ? seen : cap, ranges = (long long)x.batch * Hkv * p.nchunk;
    a.whole = rs::kv_attention_whole(p, D, fp8, most, ranges);
    a.by_length = (most > 1280 || !a.whole) && ranges > p.nwg && ranges < (1 << 22) && x.batch <= rs::KV_BY_LENGTH;
    a.nwg = p.nwg;
    a.scale_log2 = (float)((double)x.scale * 1.4426950408889634);
    const bool bf = layer->io_dtype == REPLAY_BF16;
    const auto run = bf ? (fp8 ? rs::launch_kv_attention_bf16_fp8 : rs::launch_kv_attention_bf16)
                        : (fp8 ? rs::launch_kv_attention_f16_fp8 : rs::launch_kv_attention_f16);
    return LAUNCH(run(a, p, D, (hipStream_t)stream), "paged attention");
}

replay_status replay_stream_copy(void* dst, const void* src, size_t bytes, void* stream)
{
    replay_status s;
    if ((s = check_ptr(dst, "dst")) != REPLAY_OK) return s;
    if ((s = check_ptr(src, "src")) != REPLAY_OK) return s;
    if (bytes % 16) return fail(REPLAY_ERR_ALIGN, "bytes must be a multiple of 16");
    return LAUNCH(rs::launch_stream_copy(dst, src, bytes, (hipStream_t)stream), "stream copy");
}

replay_status replay_stream_read(const void* src, size_t bytes, float* partials, void* stream)
{
    replay_status s;
    if ((s = check_ptr(src, "src")) != REPLAY_OK) return s;
    if ((s = check_ptr(partials, "partials")) != REPLAY_OK) return s;
    if (bytes % 16) return fail(REPLAY_ERR_ALIGN, "bytes must be a multiple of 16");
    return LAUNCH(rs::launch_stream_read(src, bytes, partials, (hipStream_t)stream), "stream read");
}

}  // extern "C"
