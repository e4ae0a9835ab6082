// Grouped expert routing: softmax or sigmoid scores, a per-expert balance
// bias that moves the choice but not the weights, the best groups of experts
// first, then the top k inside them, renormalised and scaled.
//
//   s_e = softmax_e(l) or 1 / (1 + exp(-l_e));   c_e = s_e + b_e
//   group value: max c of the group, or the sum of its two largest c
//   keep the topk_group best groups, then the k best c inside them
//   w   = s of the kept experts (/ their sum) * scale
//
// Without a bias experts are ranked by their logit (both scores grow with
// it).  Ties go to the lower index.  Selection values are compared in 64
// bits: a batch of 16384 tokens with 256 experts holds pairs of values closer
// than an fp32 rounding at the border of a choice, and such a pair would be
// picked by the rounding of the exponential.
#include "internal.h"

namespace moe {
namespace {

constexpr int kWave = 64;
constexpr int kWaves = 4;                        // tokens per workgroup, one per wavefront
constexpr int kPer = kMaxGroupedExperts / kWave; // experts per lane: e = lane + 64 j

// Order-preserving 64-bit key of a selection value; 0 = masked.
__device__ __forceinline__ uint64_t key64(double c) {
    if (!(c > -__builtin_huge_val())) return 0ull;   // NaN and -inf
    const uint64_t b = __builtin_bit_cast(uint64_t, c == 0.0 ? 0.0 : c);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const uint64_t o = __shfl_xor(v, d, kWave);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

template <typename LT>
__global__ __launch_bounds__(kWaves * kWave) void route_grouped_kernel(GroupedArgs a, const LT* __restrict__ logits) {
    __shared__ double val[kWaves][kMaxGroupedExperts];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int i = blockIdx.x * kWaves + wave;
    if (i >= a.B) return;   // whole wavefronts; no workgroup barrier below
    const int B_real = a.n_valid != nullptr ? min(max(*a.n_valid, 0), a.B) : a.B;
    const size_t out = static_cast<size_t>(i) * a.k;
    if (i >= B_real) {
        if (lane < a.k) {
            a.idx[out + lane] = -1;
            a.w[out + lane] = 0.0f;
        }
        return;
    }
    double s[kPer], c[kPer];
    bool live[kPer];
    double m = -__builtin_huge_val();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = lane + kWave * j;
        float l = e < a.N ? load_logit(logits + static_cast<size_t>(i) * a.N + e) : -__builtin_huge_valf();
        l = l > 3.402823466e38f ? 3.402823466e38f : l;   // +inf counts as the largest float
        live[j] = l > -__builtin_huge_valf();
        s[j] = live[j] ? static_cast<double>(l) : -__builtin_huge_val();
        m = s[j] > m ? s[j] : m;
    }
    const bool rank_by_logit = a.bias == nullptr;
#pragma unroll
    for (int j = 0; j < kPer; ++j) c[j] = s[j];
    if (a.softmax) {
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) m = fmax(m, __shfl_xor(m, d, kWave));
        double z = 0.0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            s[j] = live[j] ? exp(s[j] - m) : 0.0;
            z += s[j];
        }
        z = wave_sum(z);
#pragma unroll
        for (int j = 0; j < kPer; ++j) s[j] = z > 0.0 ? s[j] / z : 0.0;
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) s[j] = live[j] ? 1.0 / (1.0 + exp(-s[j])) : 0.0;
    }
    const int per = a.N / a.n_group;
    const bool sum2 = a.group_top2 && per > 1;
    uint64_t key[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = lane + kWave * j;
        if (!rank_by_logit && live[j]) c[j] = s[j] + static_cast<double>(a.bias[e]);
        key[j] = live[j] ? key64(c[j]) : 0ull;
        // the value that ranks groups: the score itself where two are added
        const double g = (rank_by_logit && sum2) ? s[j] : c[j];
        if (e < a.N) val[wave][e] = key[j] != 0ull ? g : -__builtin_huge_val();
    }
    if (a.n_group > 1) {
        __builtin_amdgcn_wave_barrier();
        double g = -__builtin_huge_val();
        if (lane < a.n_group) {
            double m1 = -__builtin_huge_val(), m2 = m1;
            for (int e = 0; e < per; ++e) {
                const double v = val[wave][lane * per + e];
                if (v > m1) {
                    m2 = m1;
                    m1 = v;
                } else if (v > m2) {
                    m2 = v;
                }
            }
            g = (sum2 && m2 > -__builtin_huge_val()) ? m1 + m2 : m1;
        }
        uint64_t gk = lane < a.n_group ? key64(g) : 0ull;
        uint64_t kept = 0ull;
        for (int r = 0; r < a.topk_group; ++r) {
            const uint64_t best = wave_max(gk);
            if (best == 0ull) break;
            const int o = __ffsll(static_cast<unsigned long long>(__ballot(gk == best))) - 1;
            kept |= 1ull << o;
            if (lane == o) gk = 0ull;
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (!((kept >> (min(lane + kWave * j, a.N - 1) / per)) & 1ull)) key[j] = 0ull;
    }
    // k selections; lane r keeps the r-th pick
    int pick = -1;
    double ps = 0.0;
    for (int r = 0; r < a.k; ++r) {
        uint64_t best = 0ull;
        int bj = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (key[j] > best) {
                best = key[j];
                bj = j;
            }
        const uint64_t top = wave_max(best);
        if (top == 0ull) break;
        // among the lanes that hold it, the lowest expert (e = lane + 64 j)
        int e = best == top ? lane + kWave * bj : 0x7fffffff;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) e = min(e, __shfl_xor(e, d, kWave));
        double se = 0.0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (e == lane + kWave * j) {
                key[j] = 0ull;
                se = s[j];
            }
        se = __shfl(se, e & (kWave - 1), kWave);
        if (lane == r) {
            pick = e;
            ps = se;
        }
    }
    const double sum = wave_sum(ps);
    if (a.renorm) ps = sum > 0.0 ? ps / sum : 0.0;
    if (lane < a.k) {
        a.idx[out + lane] = pick;
        a.w[out + lane] = static_cast<float>(ps * static_cast<double>(a.scale));
    }
}

}  // namespace

hipError_t launch_route_grouped(const GroupedArgs& a, hipStream_t s) {
    const unsigned grid = (a.B + kWaves - 1) / kWaves;
    if (a.logits_dtype == MOE_DT_BF16)
        route_grouped_kernel<uint16_t><<<grid, kWaves * kWave, 0, s>>>(a, static_cast<const uint16_t*>(a.logits));
    else
        route_grouped_kernel<float><<<grid, kWaves * kWave, 0, s>>>(a, static_cast<const float*>(a.logits));
    return hipGetLastError();
}

}  // namespace moe
