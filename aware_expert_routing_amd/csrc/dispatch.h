// Dispatch of routed pairs, shared by the routing kernels (device code).
#pragma once

#include "internal.h"

namespace moe {
namespace {

constexpr int kWave = 64;

// Dispatch of one workgroup: histogram, exclusive scan, (expert, token)-
// ordered permutation and the active list.  A token's position inside its
// expert's bucket is the number of lower-numbered tokens routed to the same
// expert, read off a per-expert token bitmask, so the result needs no
// ordering of atomics.  `idx` may live in LDS or in global memory.
// The dispatch's LDS: per-expert counts and token bitmasks, then offsets.
struct DispLds {
    int cnt[kMaxExperts];
    int off[kMaxExperts + 1];
    unsigned long long tokmask[kMaxExperts][kMaxBatch / 64];
};
__device__ __forceinline__ void disp_clear(DispLds& d) {
    for (int e = threadIdx.x; e < kMaxExperts; e += blockDim.x) {
        d.cnt[e] = 0;
        d.tokmask[e][0] = 0ull;
        d.tokmask[e][1] = 0ull;
    }
}
// Count the routed pair (token t, expert e) (e valid).
__device__ __forceinline__ void disp_add(DispLds& d, int t, int e) {
    atomicAdd(&d.cnt[e], 1);
    atomicOr(&d.tokmask[e][t >> 6], 1ull << (t & 63));
}

// kCounted: the caller cleared d and counted every pair with disp_add (and
// synchronised the workgroup after); otherwise this function does both.
template <bool kCounted = false>
__device__ __forceinline__ void dispatch_block(const int32_t* idx, int B, int N, int k, int32_t* cnt,
                                               int32_t* offsets, int32_t* perm, int32_t* active,
                                               int32_t* T_out, DispLds& d) {
    int* const cnt_s = d.cnt;
    int* const off_s = d.off;
    const int tid = threadIdx.x;
    const int pairs = B * k;
    if constexpr (!kCounted) {
        disp_clear(d);
        __syncthreads();
        for (int q = tid; q < pairs; q += blockDim.x) {
            const int e = idx[q];
            if (e >= 0 && e < N) disp_add(d, q / k, e);
        }
        __syncthreads();
    }
    if (tid < kWave) {
        const int lane = tid;
        const int c0 = 2 * lane < N ? cnt_s[2 * lane] : 0;
        const int c1 = 2 * lane + 1 < N ? cnt_s[2 * lane + 1] : 0;
        int sum = c0 + c1;
        int act = (c0 > 0) + (c1 > 0);
        sum = wave_incl_scan(sum);   // inclusive scans over lanes
        act = wave_incl_scan(act);
        const int excl = sum - (c0 + c1);
        const int aexcl = act - ((c0 > 0) + (c1 > 0));
        if (2 * lane < N) {
            off_s[2 * lane] = excl;
            offsets[2 * lane] = excl;
            cnt[2 * lane] = c0;
        }
        if (2 * lane + 1 < N) {
            off_s[2 * lane + 1] = excl + c0;
            offsets[2 * lane + 1] = excl + c0;
            cnt[2 * lane + 1] = c1;
        }
        const int total = __builtin_amdgcn_readlane(sum, kWave - 1);
        const int tact = __builtin_amdgcn_readlane(act, kWave - 1);
        if (lane == 0) {
            off_s[N] = total;
            offsets[N] = total;
            *T_out = tact;
        }
        int pos = aexcl;   // active list, ascending, then -1
        if (2 * lane < N && c0 > 0) active[pos++] = 2 * lane;
        if (2 * lane + 1 < N && c1 > 0) active[pos++] = 2 * lane + 1;
        for (int e = tact + lane; e < N; e += kWave) active[e] = -1;
    }
    __syncthreads();
    const int total = off_s[N];
    for (int q = tid; q < pairs; q += blockDim.x) {
        const int e = idx[q];
        if (e >= 0 && e < N) {
            const int t = q / k;
            const unsigned long long lo = d.tokmask[e][0], hi = d.tokmask[e][1];
            const int below = t < 64 ? __popcll(lo & ((1ull << t) - 1ull))
                                     : __popcll(lo) + __popcll(hi & ((1ull << (t - 64)) - 1ull));
            perm[off_s[e] + below] = q;
        }
        if (q >= total) perm[q] = -1;
    }
}

__device__ __forceinline__ void wait_vmem() {   // s_waitcnt vmcnt(0)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// The hand-off after a token-group kernel's writes: every wavefront waits
// for its stores, the barrier orders them before thread 0's count (an
// agent-scope release and, in the workgroup that completes the count,
// acquire), and that workgroup writes S_base (when given) and dispatches the
// batch from idx.  The dispatch writes T to T_out, which may be the count
// itself; with reset the count is stored back to zero afterwards.
__device__ __forceinline__ void group_dispatch_last(int32_t* __restrict__ idx, int B, int N, int k,
                                                    int32_t* __restrict__ count, bool reset,
                                                    int32_t* __restrict__ cnt, int32_t* __restrict__ offsets,
                                                    int32_t* __restrict__ perm, int32_t* __restrict__ active,
                                                    int32_t* __restrict__ T_out, uint32_t* __restrict__ mask_out,
                                                    const uint32_t* sbase) {
    __shared__ int last_s;
    __shared__ int32_t idx_l[kMaxBatch * kMaxTopK];
    __shared__ DispLds disp_l;
    const int tid = threadIdx.x;
    wait_vmem();
    __syncthreads();
    if (tid == 0)
        last_s = __hip_atomic_fetch_add(count, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                 static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    if (!last_s) return;
    if (mask_out != nullptr && tid < (N + 31) / 32) mask_out[tid] = sbase[tid];
    disp_clear(disp_l);
    __syncthreads();
    for (int q = tid; q < B * k; q += blockDim.x) {   // copy and count the routed pairs
        const int e = idx[q];
        idx_l[q] = e;
        if (e >= 0 && e < N) disp_add(disp_l, q / k, e);
    }
    __syncthreads();
    dispatch_block<true>(idx_l, B, N, k, cnt, offsets, perm, active, T_out, disp_l);
    if (reset && tid == 0) *count = 0;   // the next call's launches come after this one
}

}  // namespace
}  // namespace moe
