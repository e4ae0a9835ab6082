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
// it).  Ties go to the lower index.  The decisions are those of 64-bit
// arithmetic: a batch of 16384 tokens with 256 experts holds pairs of values
// closer than an fp32 rounding at the border of a choice, and such a pair
// would be picked by the rounding of the exponential.  They are taken in fp32
// where that is certain: every value carries a bound on its error, and a token
// with a comparison inside the bounds (one or two in a thousand: 256 experts,
// k = 8) is routed again in 64 bits by its wavefront.  All in 64 bits, 16384
// such tokens took 71 us; this way 24 (39 where exact ties are common: bf16
// logits with a bias of zeros).
//
// One wavefront per token; lane l owns the kP consecutive experts from kP l,
// so that of equal values the lowest lane, and in it the first, is the lower
// index.  A selection is a lane-local maximum over order keys and a 6-step DPP
// maximum.  A lane sorts its keys first, so that a pick moves one pointer in
// place of kP comparisons.  Group values stay in registers where a group is a
// power of two of whole lanes, and go through LDS otherwise.
//
// Bounds: a few tokens by the chain of selections (k = 8: 4.3 us for one
// token's kernel, 5.8 for 77 of 160 experts), many by the vector units: 16384
// tokens of 256 fp32 logits, 18 MB, in 24 us, 0.75 TB/s, where a copy of as
// much takes 3.7.  The dispatching form (128 tokens of 128 experts, 8.6 us) runs
// 16 tokens in a workgroup, so that few have to finish before the last one
// dispatches.
#include "dispatch.h"
#include "internal.h"

namespace moe {
namespace {

constexpr double kNegInf64 = -__builtin_huge_val();
constexpr float kNegInf = -__builtin_huge_valf();

// Order-preserving keys of selection values; 0 = masked (NaN and -inf).
__device__ __forceinline__ uint32_t key32(float c) {
    if (!(c > kNegInf)) return 0u;
    const uint32_t b = __float_as_uint(c == 0.0f ? 0.0f : c);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t key64(double c) {
    if (!(c > kNegInf64)) return 0ull;
    const uint64_t b = __builtin_bit_cast(uint64_t, c == 0.0 ? 0.0 : c);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// max(v, v moved by a DPP control); 0 where the move does not reach.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xF, true)));
}
// Maximum over the wavefront, as a scalar: quads, half rows, rows, then row
// 0 into 1 and 2 into 3, and row 1 into 2 and 3; lane 63 holds it.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max_dpp<0xB1, 0xF>(v);
    v = max_dpp<0x4E, 0xF>(v);
    v = max_dpp<0x141, 0xF>(v);
    v = max_dpp<0x140, 0xF>(v);
    v = max_dpp<0x142, 0xA>(v);
    v = max_dpp<0x143, 0xC>(v);
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), kWave - 1));
}
// Maximum of floats none of which is NaN.
template <int CTRL, int ROWS>
__device__ __forceinline__ float fmax_dpp(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, ROWS, 0xF,
                                                               false)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmax_dpp<0xB1, 0xF>(v);
    v = fmax_dpp<0x4E, 0xF>(v);
    v = fmax_dpp<0x141, 0xF>(v);
    v = fmax_dpp<0x140, 0xF>(v);
    v = fmax_dpp<0x142, 0xA>(v);
    v = fmax_dpp<0x143, 0xC>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), kWave - 1));
}
template <int CTRL>
__device__ __forceinline__ float move_dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lane_value(float v, int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
// Sum over the wavefront, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    v += move_dpp<0xB1>(v);
    v += move_dpp<0x4E>(v);
    v += move_dpp<0x141>(v);
    v += move_dpp<0x140>(v);
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
    const uint32_t hi = wave_max_u32(static_cast<uint32_t>(v >> 32));
    const uint32_t lo = wave_max_u32(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// exp(x + lo) within 2 units of fp32: x log2(e) in two pieces, the second
// applied to the result's first order.  x is held to [-100, 88], where every
// step is finite (a score that this touches is below 2^-100); there lo does not
// count (the difference of two logits that ends at -inf has none).
__device__ __forceinline__ float exp_f32(float x, float lo) {
    lo = x > -100.0f ? lo : 0.0f;
    x = fminf(fmaxf(x, -100.0f), 88.0f);
    const float y = x * 1.44269502f;                       // log2(e), fp32
    const float r = __builtin_fmaf(x, 1.44269502f, -y) + __builtin_fmaf(x, 1.92596300e-8f, lo * 1.44269502f);
    const float e = __builtin_amdgcn_exp2f(y);
    return __builtin_fmaf(e, r * 0.693147182f, e);
}

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// The kP logits of the calling lane's experts; -inf past the last expert.
template <typename LT, int kP>
__device__ __forceinline__ void load_logits(const LT* row, int N, int e0, bool wide, float (&l)[kP]) {
    struct alignas(sizeof(LT) * kP) Group { LT v[kP]; };
    if (wide) {   // rows of whole groups at aligned addresses
        if (e0 < N) {
            const Group g = *reinterpret_cast<const Group*>(row + e0);
#pragma unroll
            for (int j = 0; j < kP; ++j) l[j] = as_float(g.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kP; ++j) l[j] = kNegInf;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kP; ++j) l[j] = e0 + j < N ? as_float(row[e0 + j]) : kNegInf;
    }
}

// What a token's selection gives: lane r < k holds the r-th pick (-1: none)
// and its score, and every lane the sum of the scores.
struct Picks {
    int e;
    float s, sum;
};

// Group stage, shared by both precisions: `val` holds the experts' values in
// LDS (-inf: masked).  Lanes split into n_group bands of 1 << shift lanes
// (n_group rounded up to a power of two); every lane of band g returns group
// g's value.
template <typename F>
__device__ __forceinline__ F group_value(const F* val, const GroupedArgs& a, int per, int shift, bool sum2, int lane) {
    const F none = static_cast<F>(kNegInf64);
    const int g = lane >> shift, width = 1 << shift;
    F m1 = none, m2 = none;
    if (g < a.n_group)
        for (int e = g * per + (lane & (width - 1)); e < (g + 1) * per; e += width) {
            const F v = val[e];
            m2 = v > m1 ? m1 : (v > m2 ? v : m2);
            m1 = v > m1 ? v : m1;
        }
    for (int d = 1; d < width; d <<= 1) {
        const F o1 = __shfl_xor(m1, d, kWave), o2 = __shfl_xor(m2, d, kWave);
        const F lo = o1 > m1 ? m1 : o1, hi2 = o2 > m2 ? o2 : m2;
        m1 = o1 > m1 ? o1 : m1;
        m2 = lo > hi2 ? lo : hi2;
    }
    return (sum2 && m2 > none) ? m1 + m2 : m1;
}

// The two largest of (m1 >= m2) and of a neighbour's pair, moved by a DPP control.
template <int CTRL>
__device__ __forceinline__ void merge_dpp(float& m1, float& m2) {
    const float o1 = move_dpp<CTRL>(m1), o2 = move_dpp<CTRL>(m2);
    m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
    m1 = fmaxf(m1, o1);
}
// group_value where a group is 1 << shift whole lanes: no LDS.
template <int kP>
__device__ __forceinline__ float group_value_lanes(const float (&v)[kP], int shift, bool sum2) {
    float m1 = v[0], m2 = kNegInf;
#pragma unroll
    for (int j = 1; j < kP; ++j) {
        m2 = fmaxf(m2, fminf(m1, v[j]));
        m1 = fmaxf(m1, v[j]);
    }
    if (shift > 0) merge_dpp<0xB1>(m1, m2);
    if (shift > 1) merge_dpp<0x4E>(m1, m2);
    if (shift > 2) merge_dpp<0x141>(m1, m2);
    if (shift > 3) merge_dpp<0x140>(m1, m2);
    for (int d = 16; d < (1 << shift); d <<= 1) {
        const float o1 = __shfl_xor(m1, d, kWave), o2 = __shfl_xor(m2, d, kWave);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
    }
    return (sum2 && m2 > kNegInf) ? m1 + m2 : m1;
}

// A token in 64 bits.
template <int kP>
__device__ __forceinline__ Picks route_exact(const GroupedArgs& a, const float (&l_in)[kP], double* val, int per,
                                             int shift) {
    const int lane = threadIdx.x & (kWave - 1), e0 = kP * lane;
    const bool by_logit = a.bias == nullptr, sum2 = a.group_top2 && per > 1;
    double s[kP], c[kP];
    uint64_t key[kP];
    double m = kNegInf64;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        s[j] = static_cast<double>(l_in[j]);
        c[j] = s[j];
        m = s[j] > m ? s[j] : m;
    }
    if (a.softmax) {
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) m = fmax(m, __shfl_xor(m, d, kWave));
        double z = 0.0;
#pragma unroll
        for (int j = 0; j < kP; ++j) {
            s[j] = c[j] > kNegInf64 ? exp(c[j] - m) : 0.0;
            z += s[j];
        }
        z = wave_sum(z);
#pragma unroll
        for (int j = 0; j < kP; ++j) s[j] = z > 0.0 ? s[j] / z : 0.0;
    } else {
#pragma unroll
        for (int j = 0; j < kP; ++j) s[j] = c[j] > kNegInf64 ? 1.0 / (1.0 + exp(-c[j])) : 0.0;
    }
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const int e = e0 + j;
        if (!by_logit && c[j] > kNegInf64) c[j] = s[j] + static_cast<double>(a.bias[e]);
        key[j] = key64(c[j]);
        if (a.n_group > 1 && e < a.N) val[e] = key[j] != 0ull ? ((by_logit && sum2) ? s[j] : c[j]) : kNegInf64;
    }
    if (a.n_group > 1) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const double g = group_value(val, a, per, shift, sum2, lane);
        int rank = 0;
        for (int o = 0; o < a.n_group; ++o) {
            const double v = __shfl(g, o << shift, kWave);
            rank += v > g || (v == g && o < (lane >> shift));
        }
        const uint64_t kept = __ballot(rank < a.topk_group);
#pragma unroll
        for (int j = 0; j < kP; ++j)
            if (e0 + j >= a.N || !((kept >> ((e0 + j) / per << shift)) & 1ull)) key[j] = 0ull;
    }
    Picks out{-1, 0.0f, 0.0f};
    double ps = 0.0;
    for (int r = 0; r < a.k; ++r) {
        uint64_t best = 0ull;
        int bj = 0;
        double bs = 0.0;
#pragma unroll
        for (int j = 0; j < kP; ++j)
            if (key[j] > best) {
                best = key[j];
                bj = j;
                bs = s[j];
            }
        const uint64_t top = wave_max_u64(best);
        if (top == 0ull) break;
        const int owner = __ffsll(static_cast<unsigned long long>(__ballot(best == top))) - 1;
        const int e = kP * owner + __builtin_amdgcn_readlane(bj, owner);
        const double se = __shfl(bs, owner, kWave);
#pragma unroll
        for (int j = 0; j < kP; ++j)
            if (lane == owner && j == bj) key[j] = 0ull;
        if (lane == r) {
            out.e = e;
            ps = se;
        }
    }
    // (rounded to fp32 after the division, so that tiny scores keep their ratio)
    const double sum = wave_sum(ps);
    out.s = static_cast<float>(a.renorm ? (sum > 0.0 ? ps / sum : 0.0) : ps);
    out.sum = 1.0f;
    return out;
}

// Bounds on the fp32 values' errors: a score is within kScoreErr of the row's
// largest possible score, a sum within half a unit of its size more.
constexpr float kSigmoidErr = 0x1p-21f, kSoftmaxErr = 0x1p-19f;

// One token: the wavefront's lanes hold its logits (masked ones -inf) and
// their experts' biases.  lds: kP * 64 doubles.
template <int kP>
__device__ __forceinline__ Picks route_token(const GroupedArgs& a, const float (&l)[kP], const float (&bias)[kP],
                                             double* lds, int per, int shift, int x_shift, uint32_t per_magic,
                                             bool g_lanes) {
    const int lane = threadIdx.x & (kWave - 1), e0 = kP * lane;
    const bool by_logit = a.bias == nullptr, sum2 = a.group_top2 && per > 1;
    float* const val = reinterpret_cast<float*>(lds);       // group stage: the experts' values
    float* const score = val + kP * kWave;                  // the experts' scores
    float s[kP];
    uint32_t key[kP];
    float err;   // of a score
    if (a.softmax) {
        uint32_t km = 0u;
#pragma unroll
        for (int j = 0; j < kP; ++j) km = max(km, key32(l[j]));
        const float m = key_value(wave_max_u32(km));   // (an empty row: NaN, and every expert masked)
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < kP; ++j) {
            const float d = l[j] - m, b = d - l[j];   // l - m = d + (l - (d - b)) - (m + b), exactly
            const float e = exp_f32(d, (l[j] - (d - b)) - (m + b));
            s[j] = l[j] > kNegInf ? e : 0.0f;
            z += s[j];
        }
        const float inv = 1.0f / wave_sum(z);
#pragma unroll
        for (int j = 0; j < kP; ++j) s[j] *= inv;
        err = kSoftmaxErr * inv;
    } else {
#pragma unroll
        for (int j = 0; j < kP; ++j) {
            const float v = __builtin_amdgcn_rcpf(1.0f + exp_f32(-l[j], 0.0f));
            s[j] = l[j] > kNegInf ? v : 0.0f;
        }
        err = kSigmoidErr;
    }
    float c[kP];
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const float sum = s[j] + bias[j];
        c[j] = (by_logit || !(l[j] > kNegInf)) ? l[j] : sum;
        key[j] = key32(c[j]);
        score[e0 + j] = s[j];
    }
    bool unsure = false;
    if (a.n_group > 1) {
        float gv[kP];
#pragma unroll
        for (int j = 0; j < kP; ++j) gv[j] = key[j] != 0u ? ((by_logit && sum2) ? s[j] : c[j]) : kNegInf;
        // a group as whole lanes (bands of 1 << shift of them from lane 0), or through LDS
        float g;
        if (g_lanes) {
            g = group_value_lanes<kP>(gv, shift, sum2);
        } else {
#pragma unroll
            for (int j = 0; j < kP; ++j) val[e0 + j] = gv[j];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            g = group_value(val, a, per, shift, sum2, lane);
        }
        const int mine = lane >> shift;
        bool in;
        if (by_logit && !sum2) {   // logits: exact
            int rank = 0;
            for (int o = 0; o < a.n_group; ++o) {
                const float v = lane_value(g, o << shift);
                rank += v > g || (v == g && o < mine);
            }
            in = rank < a.topk_group;
        } else {
            // Groups surely and possibly above this one.  The margin is the same for all: a sum of two values and
            // their difference's roundings, by the largest value in size (an infinity makes all unsure).
            const bool live = g > kNegInf;
            const float margin = 4.0f * err + 0x1p-20f * wave_max(live ? __builtin_fabsf(g) : 0.0f);
            const float above = g + margin, below = g - margin;
            int sure = 0, maybe = 0;
            for (int o = 0; o < a.n_group; ++o) {
                const float v = lane_value(g, o << shift);
                sure += v > above;
                maybe += !(v < below);
            }
            in = live && maybe <= a.topk_group;   // (it counts itself)
            unsure = __any(mine < a.n_group && live && !in && sure < a.topk_group);
        }
        if (g_lanes) {   // this lane's experts are in its band's group
#pragma unroll
            for (int j = 0; j < kP; ++j) key[j] = in && e0 + j < a.N ? key[j] : 0u;
        } else {
            const uint64_t kept = __ballot(in);
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const int group = static_cast<int>((static_cast<uint32_t>(e0 + j) * per_magic) >> 20);
                if (e0 + j >= a.N || !((kept >> (group << shift)) & 1ull)) key[j] = 0u;
            }
        }
    }
    Picks out{-1, 0.0f, 0.0f};
    if (!unsure) {
        // The lane's keys in descending order, equal ones as they were, each with its expert, in LDS: a lane's best
        // is the one at its pointer, and a pick moves its owner's pointer on.
        uint32_t place[kP];
#pragma unroll
        for (int j = 0; j < kP; ++j) place[j] = j;
#pragma unroll
        for (int i = 0; i < kP - 1; ++i)
#pragma unroll
            for (int j = kP - 2; j >= i; --j) {
                const bool up = key[j + 1] > key[j];
                const uint32_t hi = max(key[j], key[j + 1]), lo = min(key[j], key[j + 1]);
                const uint32_t p = up ? place[j + 1] : place[j], q = up ? place[j] : place[j + 1];
                key[j] = hi;
                key[j + 1] = lo;
                place[j] = p;
                place[j + 1] = q;
            }
        uint32_t places = 0u;   // 4 bits each
#pragma unroll
        for (int j = 0; j < kP; ++j) places |= place[j] << (4 * j);
        uint32_t* const sorted = reinterpret_cast<uint32_t*>(val);   // [kP][64]: the lane's j-th key
        if constexpr (kP > 1) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 1; j < kP; ++j) sorted[j * kWave + lane] = key[j];
        }
        uint32_t head = key[0], pick = 0u;   // pick: lane r's r-th key, and where it was
        int from = 0, ptr = 0;
        for (int r = 0; r <= a.k; ++r) {     // the last round is for the comparison behind the loop
            const uint32_t top = wave_max_u32(head);
            if (top == 0u) break;
            const int owner = __ffsll(static_cast<unsigned long long>(__ballot(head == top))) - 1;
            const bool own = lane == owner, here = lane == r;
            const int at = __builtin_amdgcn_readlane(ptr, owner) * kWave + owner;
            pick = here ? top : pick;
            from = here ? at : from;
            ptr += own ? 1 : 0;
            const uint32_t next = ptr < kP ? sorted[min(ptr, kP - 1) * kWave + lane] : 0u;
            head = own ? next : head;
        }
        // values of neighbouring picks have to differ by more than their errors (lane r + 1 holds the next one's)
        const float v = key_value(pick), v1 = __shfl_down(v, 1, kWave);
        const uint32_t pick1 = __shfl_down(pick, 1, kWave);
        const bool close = !by_logit && lane < a.k && pick1 != 0u &&
                           !(v - v1 > 2.0f * err + 0x1p-22f * (__builtin_fabsf(v) + __builtin_fabsf(v1)));
        const bool filled = lane < a.k && pick != 0u;
        const int owner = from & (kWave - 1);
        const uint32_t p = __shfl(places, owner, kWave) >> (4 * (from >> 6));
        out.e = filled ? kP * owner + static_cast<int>(p & 15u) : -1;
        out.s = score[filled ? out.e : 0];
        // scores near the end of fp32's range lose their ratio
        unsure = __any(close || (filled && out.s < 0x1p-100f));
        out.s = filled ? out.s : 0.0f;
    }
    if (__builtin_amdgcn_readfirstlane(static_cast<int>(unsure))) return route_exact<kP>(a, l, lds, per, x_shift);
    if (a.renorm) {
        out.sum = wave_sum(out.s);
        out.s = out.sum > 0.0f ? out.s / out.sum : 0.0f;
    }
    return out;
}

// W tokens per workgroup, one per wavefront.  kDispatch: the workgroup that
// finishes last dispatches the batch (it counts in a.sync).
template <typename LT, int kP, int W, bool kDispatch>
__global__ __launch_bounds__(W* kWave) void route_grouped_kernel(GroupedArgs a, int shift, int x_shift,
                                                                 uint32_t per_magic, int flags) {
    __shared__ double lds[W][kP * kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int i = blockIdx.x * W + wave;
    const int B_real = a.n_valid != nullptr ? min(max(*a.n_valid, 0), a.B) : a.B;
    if (i < a.B) {   // whole wavefronts
        Picks p{-1, 0.0f, 0.0f};
        if (i < B_real) {
            float l[kP], bias[kP];
#pragma unroll
            for (int j = 0; j < kP; ++j) bias[j] = 0.0f;
            if (a.bias != nullptr) load_logits<float, kP>(a.bias, a.N, kP * lane, (flags & 2) != 0, bias);
            load_logits<LT, kP>(static_cast<const LT*>(a.logits) + static_cast<size_t>(i) * a.N, a.N, kP * lane,
                                (flags & 1) != 0, l);
#pragma unroll
            for (int j = 0; j < kP; ++j) {   // NaN masks; +inf counts as the largest float
                l[j] = l[j] > 3.402823466e38f ? 3.402823466e38f : l[j];
                l[j] = l[j] > kNegInf ? l[j] : kNegInf;
            }
            p = route_token<kP>(a, l, bias, lds[wave], a.N / a.n_group, shift, x_shift, per_magic, (flags & 4) != 0);
        }
        if (lane < a.k) {
            a.idx[static_cast<size_t>(i) * a.k + lane] = p.e;
            a.w[static_cast<size_t>(i) * a.k + lane] = p.s * a.scale;
        }
    }
    if constexpr (kDispatch)
        group_dispatch_last(a.idx, a.B, a.N, a.k, a.sync, true, a.cnt, a.offsets, a.perm, a.active, a.T, nullptr,
                            nullptr);
}

template <typename LT, int kP>
void launch(const GroupedArgs& a, hipStream_t s) {
    const int per = a.N / a.n_group;
    int x_shift = 6;   // lanes per group: 64 over n_group rounded up to a power of two
    while ((1 << (6 - x_shift)) < a.n_group) --x_shift;
    int shift = x_shift, g_lanes = 0;   // or a group's own lanes, where it is a power of two of whole ones
    if (per % kP == 0 && ((per / kP) & (per / kP - 1)) == 0) {
        g_lanes = 4;
        shift = __builtin_ctz(per / kP);
    }
    const uint32_t magic = ((1u << 20) + per - 1) / per;   // e / per = (e * magic) >> 20 for e < 512
    // rows of whole groups at aligned addresses: of the logits, of the bias
    const int wide = a.N % kP != 0 ? 0
                                   : (reinterpret_cast<uintptr_t>(a.logits) % (sizeof(LT) * kP) == 0 ? 1 : 0) +
                                         (reinterpret_cast<uintptr_t>(a.bias) % (sizeof(float) * kP) == 0 ? 2 : 0);
    const int flags = wide + g_lanes;
    if (a.perm != nullptr) {
        if constexpr (kP <= 2)
            route_grouped_kernel<LT, kP, 16, true>
                <<<(a.B + 15) / 16, 16 * kWave, 0, s>>>(a, shift, x_shift, magic, flags);
    } else {
        route_grouped_kernel<LT, kP, 4, false><<<(a.B + 3) / 4, 4 * kWave, 0, s>>>(a, shift, x_shift, magic, flags);
    }
}

template <typename LT>
void launch_for(const GroupedArgs& a, hipStream_t s) {
    if (a.N <= 64) launch<LT, 1>(a, s);
    else if (a.N <= 128) launch<LT, 2>(a, s);
    else if (a.N <= 256) launch<LT, 4>(a, s);
    else launch<LT, 8>(a, s);
}

}  // namespace

hipError_t launch_route_grouped(const GroupedArgs& a, hipStream_t s) {
    if (a.logits_dtype == MOE_DT_BF16) launch_for<uint16_t>(a, s);
    else launch_for<float>(a, s);
    return hipGetLastError();
}

}  // namespace moe
