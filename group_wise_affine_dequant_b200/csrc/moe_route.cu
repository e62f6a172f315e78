// The router in front of the routed experts: logits [T, E] -> the topk expert
// ids and routing weights that nv_moe_swiglu and nv_gather_qmm take.
//
//   s = softmax(z) or sigmoid(z);  c = s + bias;
//   a group's score is the sum of its group_top largest c, the topk_groups
//   best groups stay open; ids = the topk largest c among the open groups'
//   experts; w = s[ids], divided by their sum (renormalize), times scale.
//
// One warp holds one token: lane l keeps experts l * VPL .. l * VPL + VPL - 1
// in registers, so a group is a run of whole lanes for the usual power-of-two
// sizes. Every expert becomes one 32-bit key: its score's (or logit's) order with
// the low log2(VPL) bits replaced by its place in the lane. Each lane sorts its keys
// once; a pass takes the largest head of all lanes (one warp reduction) and moves
// that lane's keys up. Bound by the logits' read for many tokens (the sort and the
// passes take about as many issue slots) and by latency for few.
//
// Who is chosen is exact: scores that differ only beyond fp32, or in the bits that a
// key lacks, are not left to rounding.
//   * Without a bias both score functions grow with z, so experts (and groups
//     ranked by one score) are compared by z itself; a bf16 z keeps all its bits.
//   * With a bias, or where a group's score is a sum of two, comparisons run in
//     fp32, and every one that decides (neighbours in the chosen order, the last
//     chosen and the best refused, the groups' border) has to be further apart
//     than fp32's error.
// A token that fails this (one in some thousands) is ranked again in fp64.
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
constexpr uint32_t kNone = 0x7FFFFFFFu;

struct RouteArgs {
    const void* z;
    const float* bias;
    uint32_t* ids;
    float* w;
    int64_t T;
    int E, topk, groups, topk_groups, group_top, softmax, renormalize;
    float scale;
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
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The larger value; among equals the lower index.
__device__ __forceinline__ void warp_best(double& v, int& e) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const double v2 = __shfl_xor_sync(0xffffffffu, v, o);
        const int e2 = __shfl_xor_sync(0xffffffffu, e, o);
        if (v2 > v || (v2 == v && e2 < e)) { v = v2; e = e2; }
    }
}

__device__ __forceinline__ bool masked(float z) { return !(z > kMaskedAt); }  // also NaN

// One token ranked in fp64 by one warp; c (shared memory, E doubles) holds what
// experts are ranked by, taken and closed ones are NaN. Writes the chosen ids
// to sel. Slow and plain: few tokens come here.
template <int DT>
__device__ __noinline__ void route_fp64(const RouteArgs& a, int64_t t, double* c, int* sel) {
    const int lane = threadIdx.x & 31;
    const int64_t row = t * a.E;
    const bool pair_groups = a.groups > 1 && a.group_top == 2;
    auto logit = [&](int e) { return load_elem<DT>(a.z, row + e); };
    // without a bias the logits themselves give the order (see above)
    auto rank_by_logit = [&]() {
        for (int e = lane; e < a.E; e += 32) {
            const float z = logit(e);
            if (c[e] == c[e]) c[e] = masked(z) ? -INFINITY : static_cast<double>(fminf(z, FLT_MAX));
        }
    };
    for (int e = lane; e < a.E; e += 32) c[e] = 0.0;
    __syncwarp();
    if (!a.bias && !pair_groups) {
        rank_by_logit();
    } else {
        float m = -FLT_MAX;
        for (int e = lane; e < a.E; e += 32) {
            const float z = logit(e);
            if (!masked(z)) m = fmaxf(m, fminf(z, FLT_MAX));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double sum = 0.0;
        for (int e = lane; e < a.E; e += 32) {
            const float z = logit(e);
            double s = 0.0;
            if (!masked(z)) {
                const double zd = fminf(z, FLT_MAX);
                s = a.softmax ? exp(zd - static_cast<double>(m)) : 1.0 / (1.0 + exp(-zd));
            }
            c[e] = s;
            sum += s;
        }
        if (a.softmax) sum = warp_sum(sum);
        for (int e = lane; e < a.E; e += 32) {
            double s = c[e];
            if (a.softmax && sum > 0.0) s /= sum;
            if (a.bias) s += static_cast<double>(__ldg(a.bias + e));
            c[e] = masked(logit(e)) || s != s ? -INFINITY : s;
        }
    }
    __syncwarp();
    if (a.groups > 1) {
        const int per = a.E / a.groups;
        uint32_t open = 0;  // bit i: group lane + 32 i is open
        auto group_score = [&](int g) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int i = 0; i < per; ++i) {
                const double v = c[g * per + i];
                if (v > b1) { b2 = b1; b1 = v; } else if (v > b2) { b2 = v; }
            }
            return a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
        };
        for (int k = 0; k < a.topk_groups; ++k) {
            double v = -INFINITY;
            int g = static_cast<int>(kNone);
            for (int i = 0, j = lane; j < a.groups; ++i, j += 32) {
                if (open >> i & 1u) continue;
                const double s = group_score(j);
                if (g == static_cast<int>(kNone) || s > v) { v = s; g = j; }
            }
            warp_best(v, g);
            if (g != static_cast<int>(kNone) && (g & 31) == lane) open |= 1u << (g >> 5);
        }
        __syncwarp();
        for (int i = 0, j = lane; j < a.groups; ++i, j += 32)
            if (!(open >> i & 1u))
                for (int e = 0; e < per; ++e) c[j * per + e] = NAN;
        __syncwarp();
        if (!a.bias && pair_groups) {
            rank_by_logit();
            __syncwarp();
        }
    }
    for (int k = 0; k < a.topk; ++k) {
        double v = -INFINITY;
        int e = static_cast<int>(kNone);
        for (int j = lane; j < a.E; j += 32) {
            const double s = c[j];
            if (s != s) continue;
            if (e == static_cast<int>(kNone) || s > v) { v = s; e = j; }
        }
        warp_best(v, e);
        if (lane == 0) { sel[k] = e; c[e] = NAN; }
        __syncwarp();
    }
}

// Logits e0 .. e0 + VPL - 1 of a row, -infinity behind its end; by 16-byte loads
// (or one of 4 or 8) where whole lanes' runs keep rows aligned.
template <int DT, int VPL>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t row, int e0, float (&z)[VPL]) {
    constexpr int kSize = DT == NV_F32 ? 4 : 2, kBytes = VPL * kSize;
    if constexpr (kBytes >= 4) {
        if (a.E % VPL == 0) {
            constexpr int kWords = kBytes / 4;
            uint32_t w[kWords];
            if (e0 < a.E) {
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
                z[i] = e0 < a.E ? v : -INFINITY;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) z[i] = e0 + i < a.E ? load_elem<DT>(a.z, row + e0 + i) : -INFINITY;
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
__global__ void __launch_bounds__(32 * kWarps) moe_route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ double route_smem[];  // per warp: E doubles (the fp64 ranking)
    __shared__ int s_sel[kWarps][kMaxTopk];
    constexpr uint32_t kPlace = VPL - 1;     // a key's low bits: kPlace - (place in the lane)
    constexpr float kKeyUnits = VPL - 1.f;   // what they may cost of its value, in units
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a programmatic dependent: the logits' producer ends before any access
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.T) return;
    const int e0 = lane * VPL;
    float z[VPL];
    load_row<DT, VPL>(a, t * a.E, e0, z);
    uint32_t live = 0, real = 0;  // bit i: expert e0 + i can be chosen / exists and is not masked
    float m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (e0 + i < a.E) live |= 1u << i;
        if (!masked(z[i])) {
            real |= 1u << i;
            z[i] = fminf(z[i], FLT_MAX);
            m = fmaxf(m, z[i]);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));

    // Scores that a choice or the weights need. Renormalised softmax weights are
    // ratios of exponentials: the sum over all experts cancels.
    const bool sum_needed = a.softmax && (!a.renormalize || a.bias);
    const bool pair_groups = a.groups > 1 && a.group_top == 2;
    float inv_sum = 1.f;
    auto score = [&](int i) {  // unnormalised for softmax
        if (!(real >> i & 1u)) return 0.f;
        return a.softmax ? __expf(z[i] - m) : __fdividef(1.f, 1.f + __expf(-z[i]));
    };
    float c[VPL];  // choice scores in fp32 (bias or paired groups), else the logits
    float smax = 1.f, cmax = 0.f;
    const bool ranked = a.bias || pair_groups;
    if (sum_needed || ranked) {
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            c[i] = score(i);
            part += c[i];
        }
        if (sum_needed) {
            const float sum = warp_sum(part);
            inv_sum = sum > 0.f ? 1.f / sum : 0.f;
        }
        if (a.softmax && a.bias) smax = inv_sum;  // the largest score (1 where c is not normalised)
        if (a.bias) {
            bool odd = false;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float b = e0 + i < a.E ? __ldg(a.bias + e0 + i) : 0.f;
                c[i] = fmaf(c[i], inv_sum, b);
                cmax = fmaxf(cmax, fabsf(b));
                odd |= c[i] != c[i];
            }
            if (odd)
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (c[i] != c[i]) real &= ~(1u << i);  // a NaN bias ranks with the masked
        }
    }
    // What two fp32 scores may be apart by rounding alone. __expf(x) is off by (2 + |x|)
    // units of 2^-23 of itself.
    //   sigmoid: s (1 - s) times that stays below 1.1e-7, the quotient costs 2 units
    //   and the sum in it half of one: 3.5e-7 a score.
    //   softmax: e^x (2 + |x|) stays below 2 units of the largest, the sum over VPL
    //   experts of a lane and 32 lanes VPL + 5 halves of one, its quotient 2: all of the largest score.
    //   The bias' addition: half a unit of the sum.
    float slack = 0.f;
    if (ranked) {
#pragma unroll
        for (int o = 16; o; o >>= 1) cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, o));
        slack = kKeyUnits * 1.2e-7f * (smax + cmax) + (a.softmax ? smax * (2.f * (VPL + 16) * 1.2e-7f) : 1e-6f) + (smax + cmax) * 4.8e-7f;
    }
    bool sure = true;  // every deciding comparison is beyond fp32's error

    if (a.groups > 1) {
        const int per = a.E / a.groups;
        const int lanes = per / VPL;  // lanes per group, where a group is whole lanes
        if (per % VPL != 0 || (lanes & (lanes - 1)) != 0) {
            sure = false;  // uneven groups: ranked by the fp64 path
        } else {
            float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float v = real >> i & 1u ? (ranked ? c[i] : z[i]) : -INFINITY;
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
            const uint32_t gkey = e0 < a.E ? order_key(gs) : 0u;
            const int g = e0 / per;
            bool open = false, taken = e0 >= a.E;
            uint32_t last = 0xFFFFFFFFu;
            for (int k = 0; k < a.topk_groups; ++k) {
                last = __reduce_max_sync(0xffffffffu, taken ? 0u : gkey);
                const int first = __ffs(__ballot_sync(0xffffffffu, !taken && gkey == last)) - 1;  // the lowest group
                if (g == __shfl_sync(0xffffffffu, g, first)) open = taken = true;
            }
            if (ranked && a.topk_groups < a.groups) {
                // the border between the last open and the best closed group
                const uint32_t next = __reduce_max_sync(0xffffffffu, taken ? 0u : gkey);
                const float hi = key_value(last), lo = key_value(next);
                if (lo > -INFINITY && !(hi - lo > 2.f * slack)) sure = false;
            }
            if (!open) live = 0;
        }
    }

    // topk passes over the lanes' sorted keys: masked experts have upper bits 1, closed and missing ones are 0
    const bool by_score = a.bias != nullptr;
    int my_id[2] = {0, 0};         // this lane's slots k = lane, lane + 32
    float my_s[2] = {0.f, 0.f};
    if (sure) {
        uint32_t key[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const uint32_t upper = real >> i & 1u ? order_key(by_score ? c[i] : z[i]) & ~kPlace : VPL;
            key[i] = live >> i & 1u ? upper | (kPlace - i) : 0u;
        }
        sort_descending<0, VPL>(key);
        uint32_t prev = 0u;
        for (int k = 0;; ++k) {
            // without the places: among equals the lowest lane is next, then its lowest place
            const uint32_t top = __reduce_max_sync(0xffffffffu, key[0] | kPlace);
            if (k > 0) {  // is prev certainly before top?
                if (top <= (VPL | kPlace)) {
                    // masked or nothing left: certainly behind
                } else if (by_score) {
                    sure &= key_value(prev) - key_value(top) > slack;
                } else if (DT != NV_BF16) {
                    sure &= prev != top;
                }
            }
            if (k == a.topk) break;
            prev = top;
            const int owner = __ffs(__ballot_sync(0xffffffffu, (key[0] | kPlace) == top)) - 1;
            const uint32_t place = kPlace - (__shfl_sync(0xffffffffu, key[0], owner) & kPlace);
            if (lane == owner) {
#pragma unroll
                for (int i = 0; i + 1 < VPL; ++i) key[i] = key[i + 1];
                key[VPL - 1] = 0u;
            }
            if ((k & 31) == lane) my_id[k >> 5] = owner * VPL + static_cast<int>(place);
        }
    }
    if (!sure) {
        int* sel = s_sel[warp];
        route_fp64<DT>(a, t, route_smem + static_cast<int64_t>(warp) * a.E, sel);
        __syncwarp();
        if (lane < a.topk) my_id[0] = sel[lane];
        if (lane + 32 < a.topk) my_id[1] = sel[lane + 32];
    }

    // Weights of the chosen, from their logits. Renormalised weights are ratios,
    // so a common factor that keeps them in range is free: softmax divides by
    // the largest chosen exponential, sigmoid by e^top where all logits are negative.
    float zs[2];
    float top = -FLT_MAX;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        zs[h] = 32 * h + lane < a.topk ? load_elem<DT>(a.z, t * a.E + my_id[h]) : -INFINITY;
        if (!masked(zs[h])) {
            zs[h] = fminf(zs[h], FLT_MAX);
            top = fmaxf(top, zs[h]);
        }
    }
    float base = m;
    if (a.renormalize) {
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        base = a.softmax ? top : fminf(top, 0.f);
        inv_sum = 1.f;
    } else if (!a.softmax) {
        base = 0.f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (masked(zs[h])) continue;
        if (a.softmax)
            my_s[h] = expf(zs[h] - base) * inv_sum;
        else  // without overflow on either side
            my_s[h] = zs[h] >= 0.f ? 1.f / (1.f + expf(-zs[h])) : expf(zs[h] - base) / (1.f + expf(zs[h]));
    }
    float factor = a.scale;
    if (a.renormalize) {
        const float sum = warp_sum(my_s[0] + my_s[1]);
        factor = sum > 0.f ? a.scale / sum : 0.f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (32 * h + lane < a.topk) {
            a.ids[t * a.topk + 32 * h + lane] = static_cast<uint32_t>(my_id[h]);
            a.w[t * a.topk + 32 * h + lane] = my_s[h] * factor;
        }
    }
}

template <int DT>
cudaError_t launch(const RouteArgs& a, cudaStream_t stream) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + kWarps - 1) / kWarps), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    // every launch whose tokens may need the fp64 ranking has room for it
    const bool always_sure = DT == NV_BF16 && !a.bias && a.groups == 1;
    cfg.dynamicSmemBytes = always_sure ? 0 : sizeof(double) * kWarps * static_cast<size_t>(a.E);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    if (a.E <= 32) return cudaLaunchKernelEx(&cfg, moe_route_kernel<DT, 1>, a);
    if (a.E <= 64) return cudaLaunchKernelEx(&cfg, moe_route_kernel<DT, 2>, a);
    if (a.E <= 128) return cudaLaunchKernelEx(&cfg, moe_route_kernel<DT, 4>, a);
    if (a.E <= 256) return cudaLaunchKernelEx(&cfg, moe_route_kernel<DT, 8>, a);
    if (a.E <= 512) return cudaLaunchKernelEx(&cfg, moe_route_kernel<DT, 16>, a);
    return cudaLaunchKernelEx(&cfg, moe_route_kernel<DT, 32>, a);
}

}  // namespace

cudaError_t launch_moe_route(const void* logits, int dt, int64_t T, int E, const float* bias, int softmax,
                             int groups, int topk_groups, int group_top, int topk, int renormalize,
                             float scale, uint32_t* ids, float* weights, cudaStream_t stream) {
    const RouteArgs a{logits, bias, ids, weights, T, E, topk, groups, topk_groups, group_top, softmax,
                      renormalize, scale};
    return dt == NV_F32 ? launch<NV_F32>(a, stream) : launch<NV_BF16>(a, stream);
}

}  // namespace nvq
