// kv_pages.hip -- the page pool of the paged key/value cache: block tables, slot maps and the
// stack of free pages, kept on the device.
//
// Sequence b needs max(0, ceil((len_b + n_b) / page) - held_b) new pages.  With S_b the inclusive
// sum of these needs, its pages are the stack's entries nfree - 1 - (S_b - need_b) - i, so one
// prefix sum over the batch decides every page that a step hands out and no atomic is involved.
// A release pushes its pages in the mirrored order, which makes it the reserve's inverse.
//
// What bounds them: nothing but latency.  A step moves some kilobytes; one workgroup loads len,
// held and the mask together, scans, and writes (a few dependent trips to L2).  Only packed rows
// and releases, which can move a megabyte of entries, take a second launch over many workgroups.
// Measured: reserve 2.3 us for 8 sequences, 4.2 for 4 drafts of 512; commit 1.3 and 2.2; packed rows of
// 128 prompts of up to 8011 tokens 4.5 + 5.3; release of 128 such sequences 2.4 + 3.1.
#include "common.hpp"
#include "kv.hpp"

namespace rs {

namespace {

template <typename T>
__device__ __forceinline__ T wave_scan_inclusive(T v)
{
    const int lane = lane_id();
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
    }
    return v;
}

// Inclusive sum over the workgroup; `total` receives the whole sum.  `tmp` holds one entry per
// wave; the call ends with a barrier, so `tmp` may be used again.
template <typename T>
__device__ __forceinline__ T group_scan_inclusive(T v, T* tmp, T& total)
{
    v = wave_scan_inclusive(v);
    const int w = threadIdx.x >> 6, nw = blockDim.x >> 6;
    if (lane_id() == 63) tmp[w] = v;
    __syncthreads();
    T before = 0, all = 0;
    for (int i = 0; i < nw; ++i) {
        const T x = tmp[i];
        if (i < w) before += x;
        all += x;
    }
    __syncthreads();
    total = all;
    return v + before;
}

__device__ __forceinline__ int clamp_free(int nfree, int npages) { return min(max(nfree, 0), npages); }

}  // namespace

__global__ void kv_reset_kernel(KvPool p)
{
    const size_t n = (size_t)gridDim.x * blockDim.x;
    const size_t t = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (t < 64) p.hdr[t] = t == 0 ? p.npages : 0;
    for (size_t i = t; i < (size_t)p.plan_stride * 7; i += n) p.len[i] = 0;     // len, end, held, scratch
    for (size_t i = t; i < (size_t)p.B * p.max_pages; i += n) p.table[i] = -1;
    for (size_t i = t; i < (size_t)p.npages; i += n) p.free[i] = p.npages - 1 - (int)i;
}

// One workgroup.  PACKED: leaves old held, first page index, tokens (~n where not served) and
// first row of each sequence in the scratch arrays for kv_fill_kernel; otherwise writes the table
// entries and the step's rows itself.
template <bool PACKED>
__global__ __launch_bounds__(1024) void kv_reserve_kernel(KvPool p, int ntok, const int32_t* counts,
                                                          const uint8_t* active, int rows, int64_t* slots,
                                                          int32_t* pos, int32_t* starts)
{
    __shared__ int tmp[16];
    __shared__ long long tmpl[16];
    __shared__ int s_used;
    __shared__ uint32_t s_err;
    const int tid = threadIdx.x, ps = 1 << p.page_shift;
    const int nfree = clamp_free(p.hdr[0], p.npages);
    if (tid == 0) { s_used = 0; s_err = 0; }
    __syncthreads();
    int carry = 0;               // needs of the sequences before this pass
    long long row0 = 0;          // packed rows of the sequences before this pass
    for (int base = 0; base < p.B; base += blockDim.x) {
        const int b = base + tid;
        const bool in = b < p.B;
        const int L = in ? p.len[b] : 0, H = in ? p.held[b] : 0;
        int n = 0;
        if (in && (!active || active[b])) n = PACKED ? counts[b] : ntok;
        uint32_t err = 0;
        if (n < 0) { n = 0; err = KVERR_TOO_LONG; }
        long long start = 0;
        if (PACKED) {
            long long all;
            start = row0 + group_scan_inclusive<long long>(n, tmpl, all) - n;
            row0 += all;
        }
        const bool fits = (long long)L + n <= (long long)p.max_pages * ps && (!PACKED || start + n <= rows);
        const int need = fits && in ? max(0, ((L + n + ps - 1) >> p.page_shift) - H) : 0;
        int total;
        const int upto = carry + group_scan_inclusive<int>(need, tmp, total);
        carry += total;
        const bool given = fits && (need == 0 || upto <= nfree);
        const int got = given ? need : 0, first = upto - need;
        if (!fits) err |= KVERR_TOO_LONG;
        else if (!given) err |= KVERR_NO_PAGES;
        if (in && got > 0) atomicMax(&s_used, upto);
        if (in && err) atomicOr(&s_err, err);
        if (in) {
            p.held[b] = H + got;
            p.end[b] = given ? L + n : L;
            if (PACKED) {
                const int st = (int)min(start, 0x7fffffffLL);
                p.plan[b] = H;
                p.plan[p.plan_stride + b] = first;
                p.plan[2 * p.plan_stride + b] = given ? n : ~n;
                p.plan[3 * p.plan_stride + b] = st;
                starts[b] = st;
            } else {
                int32_t* row = p.table + (size_t)b * p.max_pages;
                for (int i = 0; i < got; ++i) row[H + i] = p.free[nfree - 1 - first - i];
                int at = -1, page = 0;
                for (int i = 0; i < ntok; ++i) {
                    const int q = L + i, pi = q >> p.page_shift;
                    const bool live = given && i < n;
                    if (live && pi != at) {
                        page = pi < H ? row[pi] : p.free[nfree - 1 - first - (pi - H)];
                        at = pi;
                    }
                    const size_t r = (size_t)i * p.B + b;
                    slots[r] = live ? ((int64_t)page << p.page_shift) + (q & (ps - 1)) : -1;
                    pos[r] = live ? q : -1;
                }
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        p.hdr[2] = nfree;
        p.hdr[0] = nfree - s_used;
        if (s_err) p.hdr[1] |= s_err;
        if (PACKED) starts[p.B] = (int)min(row0, 0x7fffffffLL);
    }
    if (!PACKED) {
        for (size_t r = (size_t)ntok * p.B + tid; r < (size_t)rows; r += blockDim.x) {
            slots[r] = -1;
            pos[r] = -1;
        }
    }
}

// Table entries and packed rows of sequence blockIdx.y; the last blockIdx.y takes the rows behind
// the last sequence.
__global__ __launch_bounds__(256) void kv_fill_kernel(KvPool p, int rows, int64_t* slots, int32_t* pos,
                                                      const int32_t* starts)
{
    const int b = blockIdx.y, step = gridDim.x * 256, t0 = blockIdx.x * 256 + threadIdx.x;
    if (b == p.B) {
        for (long long r = (long long)uload(starts + p.B) + t0; r < rows; r += step) {
            slots[r] = -1;
            pos[r] = -1;
        }
        return;
    }
    const int H = uload(p.plan + b), first = uload(p.plan + p.plan_stride + b);
    const int code = uload(p.plan + 2 * p.plan_stride + b), start = uload(p.plan + 3 * p.plan_stride + b);
    const int got = uload(p.held + b) - H, L = uload(p.len + b), nfree = uload(p.hdr + 2);
    const bool given = code >= 0;
    const int n = given ? code : ~code, ps = 1 << p.page_shift;
    int32_t* row = p.table + (size_t)b * p.max_pages;
    const int32_t* top = p.free + (nfree - 1 - first);
    for (int i = t0; i < got; i += step) row[H + i] = top[-i];
    // rows of the sequence within the arrays; counted in 64 bits, since a count may be 2^31 - 1 (not
    // served, but its rows are marked)
    const long long most = min((long long)n, (long long)rows - start);
    for (long long i = t0; i < most; i += step) {
        const long long r = start + i;
        int64_t slot = -1;
        int q = -1;
        if (given) {
            q = L + (int)i;
            const int pi = q >> p.page_shift;
            slot = ((int64_t)(pi < H ? row[pi] : top[-(pi - H)]) << p.page_shift) + (q & (ps - 1));
        }
        slots[r] = slot;
        pos[r] = q;
    }
}

__global__ __launch_bounds__(256) void kv_commit_kernel(KvPool p, const int32_t* accepted)
{
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b >= p.B) return;
    const int L = p.len[b], open = p.end[b] - L;
    int n = open;
    if (accepted) {
        n = min(max(accepted[b], 0), open);
        if (n != accepted[b]) atomicOr((uint32_t*)p.hdr + 1, KVERR_CLAMPED);
    }
    p.len[b] = L + n;
    p.end[b] = L + n;
}

// One workgroup: where each released sequence's pages go on the stack, and its empty state.
__global__ __launch_bounds__(1024) void kv_release_plan_kernel(KvPool p, const uint8_t* mask)
{
    __shared__ int tmp[16];
    const int tid = threadIdx.x;
    const int nfree = clamp_free(p.hdr[0], p.npages);
    int carry = 0;
    for (int base = 0; base < p.B; base += blockDim.x) {
        const int b = base + tid;
        const bool out = b < p.B && (!mask || mask[b]);
        const int H = out ? p.held[b] : 0;
        int total;
        const int upto = carry + group_scan_inclusive<int>(H, tmp, total);
        carry += total;
        if (b < p.B) {
            p.plan[b] = H;
            p.plan[p.plan_stride + b] = upto - H;
        }
        if (out) {
            p.len[b] = 0;
            p.end[b] = 0;
            p.held[b] = 0;
        }
    }
    __syncthreads();
    if (tid == 0) {
        p.hdr[2] = nfree + carry;
        p.hdr[0] = min(nfree + carry, p.npages);
    }
}

__global__ __launch_bounds__(256) void kv_release_kernel(KvPool p)
{
    const int b = blockIdx.y;
    const int H = uload(p.plan + b), top = uload(p.hdr + 2) - 1 - uload(p.plan + p.plan_stride + b);
    int32_t* row = p.table + (size_t)b * p.max_pages;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < H; i += gridDim.x * 256) {
        if ((unsigned)(top - i) < (unsigned)p.npages) p.free[top - i] = row[i];
        row[i] = -1;
    }
}

// Workgroups per sequence of the two-launch operations: 2048 in all, enough to fill the chip for
// one long prompt as for many short ones, and never more than the largest row could use.
static int fill_groups(const KvPool& p, long long most)
{
    const long long want = 2048 / p.B, use = (most + 255) / 256;
    return (int)(use < want ? use : want) > 1 ? (int)(use < want ? use : want) : 1;
}

static int plan_threads(int B) { return B >= 1024 ? 1024 : (B + 63) / 64 * 64; }

hipError_t launch_kv_reset(const KvPool& p, hipStream_t s)
{
    const size_t most = (size_t)p.B * p.max_pages > (size_t)p.npages ? (size_t)p.B * p.max_pages : (size_t)p.npages;
    const int groups = (int)((most + 1023) / 1024 < 1024 ? (most + 1023) / 1024 : 1024);
    hipLaunchKernelGGL(kv_reset_kernel, dim3(groups), dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_kv_reserve(const KvPool& p, int ntok, const int32_t* counts, const uint8_t* active, int rows,
                             int64_t* slots, int32_t* pos, int32_t* starts, hipStream_t s)
{
    const dim3 block(plan_threads(p.B));
    if (!counts) {
        hipLaunchKernelGGL(kv_reserve_kernel<false>, dim3(1), block, 0, s, p, ntok, counts, active, rows, slots, pos,
                           starts);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(kv_reserve_kernel<true>, dim3(1), block, 0, s, p, 0, counts, active, rows, slots, pos, starts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kv_fill_kernel, dim3(fill_groups(p, rows), p.B + 1), dim3(256), 0, s, p, rows, slots, pos,
                       starts);
    return hipGetLastError();
}

hipError_t launch_kv_commit(const KvPool& p, const int32_t* accepted, hipStream_t s)
{
    hipLaunchKernelGGL(kv_commit_kernel, dim3((p.B + 255) / 256), dim3(256), 0, s, p, accepted);
    return hipGetLastError();
}

hipError_t launch_kv_release(const KvPool& p, const uint8_t* mask, hipStream_t s)
{
    hipLaunchKernelGGL(kv_release_plan_kernel, dim3(1), dim3(plan_threads(p.B)), 0, s, p, mask);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kv_release_kernel, dim3(fill_groups(p, p.max_pages), p.B), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace rs
