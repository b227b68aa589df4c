// kv.hpp -- kernel argument blocks and launchers of the paged key/value cache (library-private).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rs {

enum : int { KV_BF16 = 0, KV_F16 = 1 };          // io element type
enum : int { KV_ROT_HALVES = 0, KV_ROT_ADJACENT = 1 };

// Error bits (mirror REPLAY_KVERR_* of the public header).
constexpr uint32_t KVERR_NO_PAGES = 0x1u, KVERR_TOO_LONG = 0x2u, KVERR_BAD_SLOT = 0x4u, KVERR_CLAMPED = 0x8u;

// The pool's region as pointers.  hdr: word 0 free pages, word 1 error bits,
// word 2 the free pages that a two-launch operation counts from.
struct KvPool {
    int B, npages, page_shift, max_pages;
    int32_t *hdr, *len, *end, *held, *plan, *table, *free;
    int plan_stride;         // words between the four scratch arrays
};
hipError_t launch_kv_reset(const KvPool& p, hipStream_t s);
hipError_t launch_kv_reserve(const KvPool& p, int ntok, const int32_t* counts, const uint8_t* active, int rows,
                             int64_t* slots, int32_t* pos, int32_t* starts, hipStream_t s);
hipError_t launch_kv_commit(const KvPool& p, const int32_t* accepted, hipStream_t s);
hipError_t launch_kv_release(const KvPool& p, const uint8_t* mask, hipStream_t s);

struct KvAppend {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int64_t* slots;
    const int32_t* pos;
    const float* freq;
    const uint8_t* axis;
    void *q_out, *K, *V;
    const float *k_scale, *v_scale;
    uint32_t* err;
    int naxes, rows, Hq, Hkv, D, page_shift, rot;
    int64_t nslots;          // npages * page_size
};
hipError_t launch_kv_append(const KvAppend& a, int io, bool fp8, int style, hipStream_t s);

struct KvAttention {
    const void* q;
    int64_t q_stride;
    const void *K, *V;
    const float *k_scale, *v_scale;
    const int32_t *table, *end;
    const uint8_t* active;
    void* o;
    float* lse;
    uint32_t* err;
    int32_t* meta;           // [nwg][2]: the split ranges, by range (first and last workgroup) where there are no
                             // more ranges than workgroups, else by the workgroup that opens one (range, last)
    float* part_ml;          // [2 nwg][rpc][2]: reference exponent and sum of each partial row
    float* part_o;           // [2 nwg][rpc][D]
    int B, Hq, Hkv, group, T, npages, page_shift, max_pages, window;
    int rows;                // T * group rows share a key/value head
    int rpc;                 // rows of a chunk, at most 16 RB RW
    int nchunk;              // chunks of rows
    bool whole;              // a workgroup per range, nothing to join
    bool by_length;          // a workgroup per range, the longest first: if whole, or if that is even enough
    int nwg;                 // workgroups of the line
    float scale_log2;        // scale * log2(e)
};
// How a call is cut: row blocks of 16 per wave, row groups (more than one in the wide kernel), rows
// of a chunk, chunks, workgroups.  The rule stands at kv_attention_plan.
struct KvPlan {
    int RB, RW;
    bool wide;
    int rpc, nchunk, nwg;
};
// Workgroups of four waves per CU where keys and values go straight to registers: two, or one where two
// would not leave a wave the registers for its outputs and the blocks on their way.  A token loop that
// spills is slower (537 MB of bf16 cache, one workgroup against two: 256 channels, 4 rows 96 / 125 us, 32
// rows 109 / 230; 128 channels, 32 rows 94 / 116); three for the narrow ones gain nothing.
constexpr int kv_occ(int D, bool fp8, int RB)
{
    return D == 256 || (D == 128 && RB == 2 && !fp8) ? 1 : 2;
}
KvPlan kv_attention_plan(int D, bool fp8, int rows);
constexpr int KV_BY_LENGTH = 1024;       // sequences that can be taken in the order of their lengths
// Whether ranges of at most `tokens` tokens are short enough for a workgroup each.
bool kv_attention_whole(const KvPlan& p, int D, bool fp8, long long tokens, long long ranges);
// One translation unit per io and cache type.
hipError_t launch_kv_attention_bf16(const KvAttention& a, const KvPlan& p, int D, hipStream_t s);
hipError_t launch_kv_attention_bf16_fp8(const KvAttention& a, const KvPlan& p, int D, hipStream_t s);
hipError_t launch_kv_attention_f16(const KvAttention& a, const KvPlan& p, int D, hipStream_t s);
hipError_t launch_kv_attention_f16_fp8(const KvAttention& a, const KvPlan& p, int D, hipStream_t s);

}  // namespace rs
