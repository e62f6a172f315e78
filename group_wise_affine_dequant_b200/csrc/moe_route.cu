// The router in front of the routed experts: logits [T, E] -> the topk expert
// ids and routing weights that nv_moe_swiglu and nv_gather_qmm take.
//
//   s = softmax(z) or sigmoid(z);  c = s + bias;
//   a group's score is the sum of its group_top largest c, the topk_groups
//   best groups stay open; ids = the topk largest c among the open groups'
//   experts; w = s[ids], divided by their sum (renormalize), times scale.
//
// One warp holds one token: lane l keeps experts l * VPL .. l * VPL + VPL - 1
// in registers; with groups, each of them starts on lanes of its own. Every expert becomes one 32-bit key: its score's (or logit's) order with
// the low log2(VPL) bits replaced by its place in the lane. Each lane sorts its keys
// once; a pass takes the largest head of all lanes (one warp reduction) and moves
// that lane's keys up. Bound by the logits' read for many tokens (the sort and the
// passes take about as many issue slots) and by latency for few: 16384 tokens of 256 experts,
// 8 groups, with a bias take 31 us (the logits' read 2.7; about 1200 instructions a token, at which
// the schedulers issue 78 % of the time, and 8 us of fp64 ranking); one token 4.5 us a call. Groups
// that are not whole runs of lanes used to be left to the fp64 ranking: 160 experts in 8 groups 94 us, now 15.
//
// Who is chosen is exact: scores that differ only beyond fp32, or in the bits that a
// key lacks, are not left to rounding.
//   * Without a bias both score functions grow with z, so experts (and groups
//     ranked by one score) are compared by z itself; a bf16 z keeps all its bits.
//   * With a bias, or where a group's score is a sum of two, comparisons run in
//     fp32, and every one that decides (neighbours in the chosen order, the last
//     chosen and the best refused, the groups' border) has to be further apart
//     than fp32's error, or of experts with the same logit and bias.
// A token that fails this (about one in a thousand of 16384 x 256 with a bias and 8 groups) is ranked again in fp64.
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "kernels.cuh"
#include "tma.cuh"

namespace nvq {
namespace {

constexpr int kWarps = 4;            // tokens per CTA
constexpr int kMaxTopk = 64;         // as nv_moe_swiglu
constexpr float kMaskedAt = -3.3895313892515355e38f;  // the lowest bf16: a logit at or below it is masked

struct RouteArgs {
    const void* z;
    const float* bias;
    uint32_t* ids;
    float* w;
    int64_t T;
    int E, topk, groups, topk_groups, group_top, softmax, renormalize;
    float scale;
    // Where experts are: a run of `per` of them on every 1 << lg_lanes lanes, VPL a lane. A run is a
    // group (by_group), or all experts on the 32 lanes.
    int per, lg_lanes;
    bool by_group;
    bool whole;  // every lane that has experts has VPL of them
    __device__ __forceinline__ int first(int lane, int vpl) const {
        return (lane >> lg_lanes) * per + (lane & ((1 << lg_lanes) - 1)) * vpl;
    }
    __device__ __forceinline__ int count(int lane, int vpl) const {
        const int left = per - (lane & ((1 << lg_lanes) - 1)) * vpl;
        return (lane >> lg_lanes) * per >= E || left <= 0 ? 0 : left < vpl ? left : vpl;
    }
};

// Order-preserving map of a float to an unsigned integer (NaN does not occur); 0 is below every value.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);  // -0 becomes +0
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A lane's n logits of a row from e0 on, -infinity behind them; by 16-byte loads
// (or one of 4 or 8) where all lanes' runs are whole and aligned.
template <int DT, int VPL>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t row, int e0, int n, float (&z)[VPL]) {
    constexpr int kSize = DT == NV_F32 ? 4 : 2, kBytes = VPL * kSize;
    if constexpr (kBytes >= 4) {
        if (a.whole) {
            constexpr int kWords = kBytes / 4;
            uint32_t w[kWords];
            if (n > 0) {
                const char* p = static_cast<const char*>(a.z) + (row + e0) * kSize;
                if constexpr (kBytes % 16 == 0) {
#pragma unroll
                    for (int i = 0; i < kWords / 4; ++i) {
                        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
                        w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
                    }
                } else if constexpr (kBytes == 8) {
                    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
                    w[0] = u.x; w[1] = u.y;
                } else {
                    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
                }
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                float v;
                if constexpr (DT == NV_F32)
                    v = __uint_as_float(w[i]);
                else
                    v = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
                z[i] = n > 0 ? v : -INFINITY;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) z[i] = i < n ? load_elem<DT>(a.z, row + e0 + i) : -INFINITY;
}

// The bias of a lane's n experts from e0 on, 0 behind them.
template <int VPL>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int e0, int n, float (&b)[VPL]) {
    if constexpr (VPL % 4 == 0) {
        if (a.whole && (reinterpret_cast<uintptr_t>(a.bias) & 15u) == 0) {
#pragma unroll
            for (int i = 0; i < VPL; i += 4) {
                const float4 u = n > 0 ? __ldg(reinterpret_cast<const float4*>(a.bias + e0 + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
                b[i] = u.x; b[i + 1] = u.y; b[i + 2] = u.z; b[i + 3] = u.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) b[i] = i < n ? __ldg(a.bias + e0 + i) : 0.f;
}

// A double's order as two words, never 0 as a pair.
__device__ __forceinline__ void order_key(double d, uint32_t& hi, uint32_t& lo) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(d + 0.0));
    const unsigned long long k = u >> 63 ? ~u : u | 0x8000000000000000ull;
    hi = static_cast<uint32_t>(k >> 32);
    lo = static_cast<uint32_t>(k);
}
// The lowest lane among those with the warp's largest (hi, lo).
__device__ __forceinline__ int best_lane(uint32_t hi, uint32_t lo) {
    const uint32_t h = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t l = __reduce_max_sync(0xffffffffu, hi == h ? lo : 0u);
    return __ffs(__ballot_sync(0xffffffffu, hi == h && lo == l)) - 1;
}

// One token ranked in fp64, experts laid out as in the kernel; the chosen go to sel.
// gs (shared memory, E + groups doubles) is for groups that are not whole lanes.
template <int DT, int VPL>
__device__ __noinline__ void route_exact(const RouteArgs& a, int64_t t, double* gs, int* sel) {
    const int lane = threadIdx.x & 31, e0 = a.first(lane, VPL), n = a.count(lane, VPL);
    const bool pair_groups = a.groups > 1 && a.group_top == 2;
    float z[VPL];
    load_row<DT, VPL>(a, t * a.E, e0, n, z);
    float m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        z[i] = fminf(z[i] > kMaskedAt ? z[i] : -INFINITY, FLT_MAX);
        m = fmaxf(m, z[i]);
    }
    double c[VPL];  // without a bias the logits themselves give the order (see above)
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = z[i];
    if (a.bias || pair_groups) {
        double part = 0.0;
        if (a.softmax) m = warp_max(m);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const double zd = z[i];
            c[i] = a.softmax ? exp(zd - static_cast<double>(m)) : 1.0 / (1.0 + exp(-zd));
            part += c[i];
        }
        const double sum = a.softmax ? warp_sum(part) : 1.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (sum > 0.0) c[i] /= sum;
            if (a.bias && i < n) c[i] += static_cast<double>(__ldg(a.bias + e0 + i));
            if (!(z[i] > -INFINITY) || c[i] != c[i]) c[i] = -INFINITY;
        }
    }
    uint32_t open = 0;  // bit i: expert e0 + i can be chosen
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (i < n) open |= 1u << i;
    if (a.groups > 1) {
        const int per = a.E / a.groups, lanes = 1 << a.lg_lanes;
        if (a.by_group) {
            double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                b2 = fmax(b2, fmin(b1, c[i]));
                b1 = fmax(b1, c[i]);
            }
            for (int o = 1; o < lanes; o <<= 1) {
                const double o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
                b2 = fmax(fmax(b2, o2), fmin(b1, o1));
                b1 = fmax(b1, o1);
            }
            uint32_t hi = 0, lo = 0;
            if (e0 < a.E && (lane & (lanes - 1)) == 0) order_key(pair_groups && b2 > -INFINITY ? b1 + b2 : b1, hi, lo);
            const int first = lane & ~(lanes - 1);
            bool chosen = false;
            for (int k = 0; k < a.topk_groups; ++k) {
                if (best_lane(hi, lo) == first) {
                    chosen = true;
                    hi = lo = 0;
                }
            }
            if (!chosen) open = 0;
        } else {
            double* cs = gs + a.groups;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i < n) cs[e0 + i] = c[i];
            __syncwarp();
            for (int g = 0; g < a.groups; ++g) {
                double b1 = -INFINITY, b2 = -INFINITY;
                for (int i = lane; i < per; i += 32) {
                    const double v = cs[g * per + i];
                    b2 = fmax(b2, fmin(b1, v));
                    b1 = fmax(b1, v);
                }
                for (int o = 16; o; o >>= 1) {
                    if (o >= per) continue;  // those lanes hold nothing
                    const double o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
                    b2 = fmax(fmax(b2, o2), fmin(b1, o1));
                    b1 = fmax(b1, o1);
                }
                if (lane == 0) gs[g] = pair_groups && b2 > -INFINITY ? b1 + b2 : b1;
            }
            __syncwarp();
            for (int k = 0; k < a.topk_groups; ++k) {  // the chosen become NaN
                uint32_t hi = 0, lo = 0;
                int g = 0;
                for (int j = lane; j < a.groups; j += 32) {
                    uint32_t h = 0, l = 0;
                    if (gs[j] == gs[j]) order_key(gs[j], h, l);
                    if (h > hi || (h == hi && l > lo)) { hi = h; lo = l; g = j; }
                }
                // among equals the lowest group, which need not be the lowest lane's
                const uint32_t h = __reduce_max_sync(0xffffffffu, hi);
                const uint32_t l = __reduce_max_sync(0xffffffffu, hi == h ? lo : 0u);
                g = static_cast<int>(__reduce_min_sync(0xffffffffu, hi == h && lo == l ? static_cast<uint32_t>(g) : 0x7FFFFFFFu));
                if (lane == 0) gs[g] = NAN;
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i < n && gs[(e0 + i) / per] == gs[(e0 + i) / per]) open &= ~(1u << i);
        }
    }
    if (!a.bias && pair_groups) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = z[i];
    }
    for (int k = 0; k < a.topk; ++k) {
        uint32_t hi = 0, lo = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            uint32_t h = 0, l = 0;
            if (open >> i & 1u) order_key(c[i], h, l);
            if (h > hi || (h == hi && l > lo)) { hi = h; lo = l; at = i; }
        }
        const int owner = best_lane(hi, lo);
        if (lane == owner) {
            sel[k] = e0 + at;
            open &= ~(1u << at);
        }
    }
    __syncwarp();
}

// Descending sort of N registers (Batcher's odd-even merge sort).
__device__ __forceinline__ void order_pair(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b), lo = min(a, b);
    a = hi;
    b = lo;
}
template <int LO, int N, int R, int V>
__device__ __forceinline__ void merge_descending(uint32_t (&k)[V]) {
    if constexpr (2 * R < N) {
        merge_descending<LO, N, 2 * R>(k);
        merge_descending<LO + R, N, 2 * R>(k);
#pragma unroll
        for (int i = LO + R; i + R < LO + N; i += 2 * R) order_pair(k[i], k[i + R]);
    } else {
        order_pair(k[LO], k[LO + R]);
    }
}
template <int LO, int N, int V>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[V]) {
    if constexpr (N > 1) {
        sort_descending<LO, N / 2>(k);
        sort_descending<LO + N / 2, N / 2>(k);
        merge_descending<LO, N, 1>(k);
    }
}
// The float a key came from.
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// VPL: experts per lane. 32 * VPL >= E.
template <int DT, int VPL>
__global__ void __launch_bounds__(32 * kWarps, VPL <= 8 ? 12 : 1) moe_route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ double route_smem[];  // per warp: E + groups doubles (the fp64 ranking)
    __shared__ int s_sel[kWarps][kMaxTopk];
    constexpr uint32_t kPlace = VPL - 1;     // a key's low bits: kPlace - (place in the lane)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a programmatic dependent: the logits' producer ends before any access
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.T) return;
    const int e0 = a.first(lane, VPL), n = a.count(lane, VPL);
    float z[VPL];
    load_row<DT, VPL>(a, t * a.E, e0, n, z);
    // a masked expert's logit becomes -infinity: its score is 0, its rank last
    float m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        z[i] = fminf(z[i] > kMaskedAt ? z[i] : -INFINITY, FLT_MAX);
        m = fmaxf(m, z[i]);
    }
    if (a.softmax) m = warp_max(m);

    // Scores that a choice or the weights need. Renormalised softmax weights are
    // ratios of exponentials: the sum over all experts cancels.
    const bool by_score = a.bias != nullptr;
    const bool pair_groups = a.groups > 1 && a.group_top == 2;
    const bool ranked = by_score || pair_groups;
    float inv_sum = 1.f;
    float c[VPL];     // choice scores in fp32 (-infinity: masked)
    float slack = 0.f;
    if (a.softmax) {
        if (ranked || !a.renormalize) {
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                c[i] = __expf(z[i] - m);
                part += c[i];
            }
            if (by_score || !a.renormalize) {
                const float sum = warp_sum(part);
                inv_sum = sum > 0.f ? 1.f / sum : 0.f;
            }
        }
    } else if (ranked) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = rcp_approx(1.f + __expf(-z[i]));
    }
    if (ranked) {
        float smax = a.softmax && by_score ? inv_sum : 1.f;  // the largest score
        float cmax = 0.f;
        if (by_score) {
            float b[VPL];
            load_bias<VPL>(a, e0, n, b);
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                c[i] = fmaf(c[i], inv_sum, b[i]);
                cmax = fmaxf(cmax, fabsf(b[i]));
            }
            cmax = warp_max(cmax);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = z[i] > -INFINITY && c[i] == c[i] ? c[i] : -INFINITY;  // a NaN bias too
        // What two fp32 scores may be apart by rounding alone. __expf(x) is off by (2 + |x|)
        // units of 2^-23 of itself.
        //   sigmoid: s (1 - s) times that stays below 1.1e-7, the reciprocal costs a unit
        //   and the sum in it half of one: 3.5e-7 a score.
        //   softmax: e^x (2 + |x|) stays below 2 units of the largest, the sum over VPL
        //   experts of a lane and 32 lanes VPL + 5 halves of one, its quotient 2: all of the largest score.
        //   The bias' addition: half a unit of the sum. The bits a key lacks: VPL - 1 units of it.
        slack = (VPL + 3) * 1.2e-7f * (smax + cmax) + (a.softmax ? smax * (2.f * (VPL + 16) * 1.2e-7f) : 1e-6f);
    }
    bool sure = true;  // every deciding comparison is beyond fp32's error

    bool open = n > 0;  // this lane's experts can be chosen
    if (a.groups > 1) {
        const int lanes = 1 << a.lg_lanes;
        if (!a.by_group) {
            sure = false;  // more groups than lanes, or too large ones: ranked by the fp64 path
        } else {
            float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float v = ranked ? c[i] : z[i];
                b2 = fmaxf(b2, fminf(b1, v));
                b1 = fmaxf(b1, v);
            }
            for (int o = 1; o < lanes; o <<= 1) {
                const float o1 = __shfl_xor_sync(0xffffffffu, b1, o);
                const float o2 = __shfl_xor_sync(0xffffffffu, b2, o);
                b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
                b1 = fmaxf(b1, o1);
            }
            const float gs = pair_groups && b2 > -INFINITY ? b1 + b2 : b1;
            const int first = lane & ~(lanes - 1);  // the group's first lane, which has its key (0: taken or not there)
            uint32_t gkey = lane == first && open ? order_key(gs) : 0u;
            open = false;
            uint32_t last = 0u;
            for (int k = 0; k < a.topk_groups; ++k) {
                last = __reduce_max_sync(0xffffffffu, gkey);
                if (first == __ffs(__ballot_sync(0xffffffffu, gkey == last)) - 1) {  // the lowest such group
                    open = n > 0;
                    gkey = 0u;
                }
            }
            if (ranked && a.topk_groups < a.groups) {
                // the border between the last open and the best closed group
                const uint32_t next = __reduce_max_sync(0xffffffffu, gkey);
                const float hi = key_value(last), lo = key_value(next);
                if (lo > -INFINITY && !(hi - lo > 2.f * slack)) sure = false;
            }
        }
    }

    // topk passes over the lanes' sorted keys; closed and missing experts are 0
    int id0 = 0, id1 = 0;          // the chosen of this lane's slots k = lane and lane + 32
    if (sure) {
        constexpr uint32_t kLast = 0x007FFFFFu | kPlace;  // -infinity's key: behind it nothing is left to tell apart
        uint32_t key[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const uint32_t k = order_key(by_score ? c[i] : z[i]);
            key[i] = open ? (k & ~kPlace) | (kPlace - i) : 0u;
        }
        if (!a.whole) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = i < n ? key[i] : 0u;
        }
        sort_descending<0, VPL>(key);
        uint32_t prev = 0u;
        float prev_value = INFINITY;
        int prev_e = 0;
        for (int k = 0;; ++k) {
            // without the places: among equals the lowest lane is next, then its lowest place
            const uint32_t top = __reduce_max_sync(0xffffffffu, key[0] | kPlace);
            const int owner = __ffs(__ballot_sync(0xffffffffu, (key[0] | kPlace) == top)) - 1;
            const int e = a.first(owner, VPL) + static_cast<int>(kPlace - (__shfl_sync(0xffffffffu, key[0], owner) & kPlace));
            if (top > kLast) {  // is the expert before certainly before this one?
                if (by_score) {
                    const float value = key_value(top);
                    if (!(prev_value - value > slack))  // the same logit and bias: the same score, in order of the ids
                        sure &= k > 0 && load_elem<DT>(a.z, t * a.E + e) == load_elem<DT>(a.z, t * a.E + prev_e) &&
                                __ldg(a.bias + e) == __ldg(a.bias + prev_e);
                    prev_value = value;
                    prev_e = e;
                } else if (DT != NV_BF16) {
                    sure &= prev != top;
                    prev = top;
                }
            }
            if (k == a.topk) break;
            if (lane == owner) {
#pragma unroll
                for (int i = 0; i + 1 < VPL; ++i) key[i] = key[i + 1];
                key[VPL - 1] = 0u;
            }
            if (k == lane) id0 = e;
            if (k == lane + 32) id1 = e;
        }
    }
    if (!sure) {
        int* sel = s_sel[warp];
        route_exact<DT, VPL>(a, t, route_smem + warp * (a.E + a.groups), sel);
        __syncwarp();
        if (lane < a.topk) id0 = sel[lane];
        if (lane + 32 < a.topk) id1 = sel[lane + 32];
    }

    // Weights of the chosen, from their logits. Renormalised weights are ratios,
    // so a common factor that keeps them in range is free: softmax divides by
    // the largest chosen exponential, sigmoid by e^top where all logits are negative.
    const bool has0 = lane < a.topk, has1 = lane + 32 < a.topk;
    float z0 = has0 ? load_elem<DT>(a.z, t * a.E + id0) : -INFINITY;
    float z1 = has1 ? load_elem<DT>(a.z, t * a.E + id1) : -INFINITY;
    z0 = fminf(z0 > kMaskedAt ? z0 : -INFINITY, FLT_MAX);
    z1 = fminf(z1 > kMaskedAt ? z1 : -INFINITY, FLT_MAX);
    float base = a.softmax ? m : 0.f;
    if (a.renormalize) {
        const float top = warp_max(fmaxf(fmaxf(z0, z1), -FLT_MAX));
        base = a.softmax ? top : fminf(top, 0.f);
        inv_sum = 1.f;
    }
    auto weight = [&](float x) {
        if (!(x > -INFINITY)) return 0.f;
        if (a.softmax) return expf(x - base) * inv_sum;
        return x >= 0.f ? 1.f / (1.f + expf(-x)) : expf(x - base) / (1.f + expf(x));  // overflows on neither side
    };
    const float s0 = weight(z0), s1 = a.topk > 32 ? weight(z1) : 0.f;
    float factor = a.scale;
    if (a.renormalize) {
        const float sum = warp_sum(s0 + s1);
        factor = sum > 0.f ? a.scale / sum : 0.f;
    }
    if (has0) {
        a.ids[t * a.topk + lane] = static_cast<uint32_t>(id0);
        a.w[t * a.topk + lane] = s0 * factor;
    }
    if (has1) {
        a.ids[t * a.topk + 32 + lane] = static_cast<uint32_t>(id1);
        a.w[t * a.topk + 32 + lane] = s1 * factor;
    }
}

template <int DT>
cudaError_t launch(const RouteArgs& a, int vpl, cudaStream_t stream) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + kWarps - 1) / kWarps), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    // every launch whose tokens may need the fp64 ranking has room for it
    const bool always_sure = DT == NV_BF16 && !a.bias && a.groups == 1;
    cfg.dynamicSmemBytes = always_sure ? 0 : sizeof(double) * kWarps * static_cast<size_t>(a.E + a.groups);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    auto kernel = vpl == 1   ? moe_route_kernel<DT, 1>
                  : vpl == 2 ? moe_route_kernel<DT, 2>
                  : vpl == 4 ? moe_route_kernel<DT, 4>
                  : vpl == 8 ? moe_route_kernel<DT, 8>
                  : vpl == 16 ? moe_route_kernel<DT, 16>
                              : moe_route_kernel<DT, 32>;
    // up to 64 KB (1023 experts, each a group); beyond what every launch may ask for, with the 1 KB of s_sel beside it
    constexpr size_t kStatic = sizeof(int) * kWarps * kMaxTopk, kFree = 48 * 1024;
    if (cfg.dynamicSmemBytes + kStatic > kFree) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(cfg.dynamicSmemBytes));
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_moe_route(const void* logits, int dt, int64_t T, int E, const float* bias, int softmax,
                             int groups, int topk_groups, int group_top, int topk, int renormalize,
                             float scale, uint32_t* ids, float* weights, cudaStream_t stream) {
    RouteArgs a{logits, bias, ids, weights, T, E, topk, groups, topk_groups, group_top, softmax, renormalize, scale,
                E, 5, false, false};
    // Each group gets a power of two of lanes, as many as there are, if they hold it with 32 experts a
    // lane; other groups (and more than 32) are found in shared memory by the fp64 ranking.
    if (groups > 1 && groups <= 32) {
        int lg = 4;
        while ((groups << lg) > 32) --lg;
        if (E / groups <= 32 << lg) {
            a.per = E / groups;
            a.lg_lanes = lg;
            a.by_group = true;
        }
    }
    int vpl = 1;
    while (vpl << a.lg_lanes < a.per) vpl *= 2;
    a.whole = a.per % vpl == 0 && E % vpl == 0;
    return dt == NV_F32 ? launch<NV_F32>(a, vpl, stream) : launch<NV_BF16>(a, vpl, stream);
}

}  // namespace nvq
