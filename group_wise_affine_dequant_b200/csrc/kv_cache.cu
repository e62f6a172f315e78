// The paged 8-bit key/value cache: writing a step's keys and values into it
// (nv_kv_quantize) and reading them back (nv_kv_dequantize).
//
// One fp32 scale per (page, head): scale = amax / 127 (int8) or amax / 448
// (E4M3) of what the block holds; a code is the representable value nearest to
// x / scale (ties to even), exactly: the quotient's rounding never decides.
// Tokens appended to a part-filled block keep its scale unless they need a
// larger one; then the codes already there are read, scaled by old / new and
// rounded again through a 256-entry table (a code has only 256 values).
//
// Both kernels: one CTA per block of tokens and run of planes (a plane is K or V of
// one head). Writing, a plane's new values stay in registers between the maximum
// and the codes, so they are read once; a few tokens (a decoding step) take one
// warp a plane, whole blocks the CTA. Bound by memory: 2 bytes in and 1 out per
// bf16 value, and the reverse for the read-back.
#include <cfloat>
#include <cstdint>

#include "kv.cuh"
#include "tma.cuh"

namespace nvq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kKeep = 4;  // 8-value chunks a thread keeps: a block of 64 tokens of 128 values

// Eight values as they are stored.
template <int DT>
struct Raw8;
template <>
struct Raw8<NV_BF16> {
    uint4 u;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    }
    __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float get(int j) const {
        const uint32_t w = j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w;
        return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
    }
    // largest magnitude's bits as fp32 bits (NaN and infinity above every number)
    __device__ __forceinline__ uint32_t most() const {
        const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                                    __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
        return max(m << 16, m & 0xFFFF0000u);
    }
};
template <>
struct Raw8<NV_F32> {
    uint4 u[2];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        u[0] = __ldg(q);
        u[1] = __ldg(q + 1);
    }
    __device__ __forceinline__ void clear() { u[0] = u[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float get(int j) const {
        const uint4& w = u[j >> 2];
        const int k = j & 3;
        return __uint_as_float(k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w);
    }
    __device__ __forceinline__ uint32_t most() const {
        uint32_t m = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            m = max(m, max(max(u[h].x & 0x7FFFFFFFu, u[h].y & 0x7FFFFFFFu), max(u[h].z & 0x7FFFFFFFu, u[h].w & 0x7FFFFFFFu)));
        return m;
    }
};

// int8: the integer nearest to x / s (ties to even), |x / s| <= 127.5. A first guess
// c by the reciprocal is off by at most one, and the remainder x - c s is exact in
// fp32 (both are multiples of s's unit, below 2 s): the guess stands where it is below s / 2.
// kMagic + c holds c in its low byte.
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
__device__ __forceinline__ uint32_t int8_exact(float x, float s, float inv) {
    float t = fmaf(x, inv, kMagic);
    const float e = fmaf(-(t - kMagic), s, x), half = 0.5f * s;
    const bool odd = __float_as_uint(t) & 1u;
    if (fabsf(e) > half || (fabsf(e) == half && odd)) t += copysignf(1.f, e);
    return __float_as_uint(t);
}

// E4M3: x / s as a float that rounds as the exact quotient does: only a quotient
// that landed on a 5-bit value (a tie's place) by rounding is moved off it, by one
// unit towards the exact value.
__device__ __forceinline__ float e4m3_exact(float x, float s) {
    const float q = __fdiv_rn(x, s);
    if ((__float_as_uint(q) & 0x3FFFFu) == 0u) {
        const float r = fmaf(-q, s, x);
        if (r != 0.f && q != 0.f)
            return __uint_as_float(__float_as_uint(q) + ((r > 0.f) == (q > 0.f) ? 1u : 0xFFFFFFFFu));
    }
    return q;
}

// Eight codes. The quick form settles all but what lies next to a tie, which is rare
// enough to be asked once for the eight: an E4M3 quotient by the reciprocal (two
// units off at most) rounds as the exact one unless its low 20 bits are within 4 of a
// half, or it is small enough for E4M3's subnormals.
template <int MODE>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float s, float inv) {
    uint32_t w[2];
    if constexpr (MODE == NV_KV_INT8) {
        uint32_t t[8];
        bool near = false;
        const float half = 0.5f * s;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fmaf(x[j], inv, kMagic);
            near |= fabsf(fmaf(-(m - kMagic), s, x[j])) >= half;
            t[j] = __float_as_uint(m);
        }
        if (near) {
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = int8_exact(x[j], s, inv);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = __byte_perm(__byte_perm(t[4 * h], t[4 * h + 1], 0x0040), __byte_perm(t[4 * h + 2], t[4 * h + 3], 0x0040), 0x5410);
    } else {
        float q[8];
        bool near = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            q[j] = x[j] * inv;
            const uint32_t u = __float_as_uint(q[j]);
            near |= (u - 0x7FFFCu & 0xFFFFFu) <= 8u || (u & 0x7FFFFFFFu) - 1u < 0x3C800000u - 1u;  // 2^-6, zero is exact
        }
        if (near) {
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = e4m3_exact(x[j], s);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h], q[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h + 2], q[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | (hi << 16);
        }
    }
    return make_uint2(w[0], w[1]);
}

// A code of the old scale as a code of the larger new one: the nearest to the
// exact c * old / new. In fp64 the product is exact and the quotient never
// rounds onto a tie that it is not on (both scales have 24 bits).
template <int MODE>
__device__ __forceinline__ uint8_t recode(uint32_t byte, float old_scale, float new_scale) {
    const double q = static_cast<double>(code_value<MODE>(byte)) * old_scale / new_scale;
    if constexpr (MODE == NV_KV_INT8) {
        return static_cast<uint8_t>(static_cast<int8_t>(__double2int_rn(q)));
    } else {
        // to fp32 by rounding to odd, which E4M3's rounding cannot tell from the exact value
        float f = __double2float_rz(q);
        if (static_cast<double>(f) != q) f = __uint_as_float(__float_as_uint(f) | 1u);
        return static_cast<uint8_t>(__nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3));
    }
}

// The block of tokens a CTA works on: sequence, page and this step's slots in it.
struct BlockWork {
    int page;          // the table's entry, not yet looked at (page_ok); -1: nothing to do
    int slot0, slot1;  // the step's tokens in the block
    int64_t row0;      // row of slot0
    bool any;          // the block has tokens of the step
};
__device__ __forceinline__ BlockWork block_work(const KvCache& c, const KvSteps& st, const SeqSpan& span, int s,
                                                int64_t j) {
    BlockWork w{};
    w.page = -1;
    const int first = span.first < 0 ? 0 : span.first;
    const int64_t b = first / c.block + j;
    if (j < 0 || span.n == 0 || b * c.block >= span.len) return w;
    const int base = static_cast<int>(b * c.block);
    w.any = true;
    w.slot0 = first > base ? first - base : 0;
    w.slot1 = span.len - base < c.block ? span.len - base : c.block;
    w.row0 = span.row0 + (base + w.slot0 - span.first);
    w.page = __ldg(st.pages + static_cast<int64_t>(s) * st.max_pages + b);
    return w;
}
// Kept apart from the lookup, so that a block's values are on their way before its page is known.
__device__ __forceinline__ bool page_ok(const KvCache& c, const KvSteps& st, const BlockWork& w) {
    if (w.page >= 0 && w.page < c.P) return true;
    if (st.flags) atomicOr(st.flags, NV_FLAG_PAGE_OUT_OF_RANGE);
    return false;
}

// i / d for 0 <= i < 2^16, by one multiplication: magic = 2^32 / d rounded up, which is
// exact there since i times its error (below d / 2^32 a unit) stays under 1 / d.
struct Divider {
    uint32_t d, magic;
    explicit Divider(uint32_t n) : d(n), magic(n == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + n - 1) / n)) {}
    __device__ __forceinline__ int of(int i) const { return d == 1 ? i : static_cast<int>(__umulhi(i, magic)); }
};

struct QuantArgs {
    const void* x[2];  // k, v
    int64_t stride[2];
    int planes;        // planes a CTA takes
    Divider vecs;      // 8-value chunks a token
    KvCache c;
    KvSteps st;
};

// One plane of a block by a team of threads (a warp or the CTA); `most` finds the
// team's maximum and is a barrier for it.
template <int DT, int MODE, class Most, class Sync>
__device__ __forceinline__ void quantize_plane(const QuantArgs& a, const BlockWork& w, int plane, int rank, int size,
                                               uint8_t* table, const Most& team_most, const Sync& sync) {
    const KvCache& c = a.c;
    const int which = plane & 1, h = plane >> 1;
    const int vecs = c.D / 8;
    const int chunks = (w.slot1 - w.slot0) * vecs;
    const void* x = which ? a.x[1] : a.x[0];
    const int64_t stride = which ? a.stride[1] : a.stride[0];
    const int64_t x0 = w.row0 * stride + static_cast<int64_t>(h) * c.D;
    auto place = [&](int i) {  // chunk i's first value
        const int tok = a.vecs.of(i);
        return x0 + tok * stride + (i - tok * vecs) * 8;
    };
    Raw8<DT> keep[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        keep[k].clear();
        if (rank + k * size < chunks) keep[k].load(x, place(rank + k * size));
    }
    if (!page_ok(c, a.st, w)) return;  // the same for the whole team
    const int64_t at = static_cast<int64_t>(w.page) * c.H + h;
    uint8_t* codes = (which ? c.v_codes : c.k_codes) + at * (static_cast<int64_t>(c.block) * c.D);
    float* scale_at = (which ? c.v_scales : c.k_scales) + at;
    const float old = w.slot0 > 0 ? *scale_at : 0.f;
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) most = max(most, keep[k].most());
    for (int i = rank + kKeep * size; i < chunks; i += size) {
        Raw8<DT> r;
        r.load(x, place(i));
        most = max(most, r.most());
    }
    most = team_most(most);
    const bool odd = most >= 0x7F800000u;  // NaN or infinities among the values: the maximum of the others
    if (odd) {
        most = 0;
        for (int i = rank; i < chunks; i += size) {
            Raw8<DT> r;
            r.load(x, place(i));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = __float_as_uint(r.get(j)) & 0x7FFFFFFFu;
                if (u < 0x7F800000u) most = max(most, u);
            }
        }
        sync();
        most = team_most(most);
    }
    constexpr float kLargest = MODE == NV_KV_INT8 ? kInt8Max : kE4m3Max;
    const float scale = fmaxf(old, __fdiv_rn(__uint_as_float(most), kLargest));
    if (rank == 0) *scale_at = scale;

    if (w.slot0 > 0 && scale > old) {  // the same for the whole team
        sync();  // the previous plane's reads of the table
        for (int i = rank; i < 256; i += size) table[i] = recode<MODE>(i, old, scale);
        sync();
        uint4* words = reinterpret_cast<uint4*>(codes);
        for (int i = rank; i < w.slot0 * c.D / 16; i += size) {
            uint4 u = words[i];
            uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = table[v[k] & 255u] | (table[v[k] >> 8 & 255u] << 8) | (table[v[k] >> 16 & 255u] << 16) |
                       (static_cast<uint32_t>(table[v[k] >> 24]) << 24);
            words[i] = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }

    // a tiny scale's reciprocal or remainders would leave the normal range: move both by 2^64, exactly
    const float lift = scale < 8.6736174e-19f ? 18446744073709551616.f : 1.f;  // 2^-60, 2^64
    const float s2 = scale * lift, inv = scale > 0.f ? 1.f / s2 : 0.f;
    const float edge = fminf(kLargest * scale, FLT_MAX);  // the product may round to infinity
    auto store = [&](const Raw8<DT>& r, int i) {
        uint2 o = make_uint2(0u, 0u);
        if (scale > 0.f) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = r.get(j);
            // NaN is kept as 0, an infinity as the largest code; so is what a subnormal scale, of a few
            // bits, leaves above it
            if (odd || lift != 1.f) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    f[j] = f[j] == f[j] ? f[j] : 0.f;
                    f[j] = fminf(fmaxf(f[j], -edge), edge);
                }
            }
            if (lift != 1.f) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] *= lift;
            }
            o = encode8<MODE>(f, s2, inv);
        }
        // the block's new slots follow one another in the page: chunk i of them is 8 bytes on
        *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(w.slot0) * c.D + 8 * static_cast<int64_t>(i)) = o;
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
        if (rank + k * size < chunks) store(keep[k], rank + k * size);
    for (int i = rank + kKeep * size; i < chunks; i += size) {
        Raw8<DT> r;
        r.load(x, place(i));
        store(r, i);
    }
}

template <int DT, int MODE>
__global__ void __launch_bounds__(kThreads, 3) kv_quantize_kernel(const __grid_constant__ QuantArgs a) {
    __shared__ uint32_t warp_most[2][kWarps];
    __shared__ uint8_t table[kWarps][256];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = kv_find_seq(a.st, blockIdx.x, 1, a.c.block, 2);
    const SeqSpan span = seq_span(a.st, s, a.c.block);
    const BlockWork w = block_work(a.c, a.st, span, s, static_cast<int64_t>(blockIdx.x) - kv_first_item(a.st, s, 1, a.c.block, 2));
    if (!w.any) return;
    const int p0 = blockIdx.y * a.planes;
    const int p1 = p0 + a.planes < 2 * a.c.H ? p0 + a.planes : 2 * a.c.H;
    if ((w.slot1 - w.slot0) * (a.c.D / 8) <= 32 * kKeep) {
        for (int p = p0 + warp; p < p1; p += kWarps)
            quantize_plane<DT, MODE>(a, w, p, lane, 32, table[warp],
                                     [](uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }, [] { __syncwarp(); });
    } else {
        int turn = 0;  // two buffers: one barrier a maximum is enough
        for (int p = p0; p < p1; ++p) {
            quantize_plane<DT, MODE>(
                a, w, p, threadIdx.x, kThreads, table[0],
                [&](uint32_t v) {
                    v = __reduce_max_sync(0xffffffffu, v);
                    turn ^= 1;
                    if (lane == 0) warp_most[turn][warp] = v;
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) v = max(v, warp_most[turn][i]);
                    return v;
                },
                [] { __syncthreads(); });
        }
    }
}

// Four codes as floats (exact).
template <int MODE>
__device__ __forceinline__ void word_values(uint32_t w, float* f) {
    if constexpr (MODE == NV_KV_INT8) {
        w ^= 0x80808080u;  // c + 128
#pragma unroll
        for (int i = 0; i < 4; ++i)  // under the mantissa of 2^23
            f[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | i)) - 8388736.f;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2_raw v = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h)), __NV_E4M3);
            const float2 x = __half22float2(__half2(v));
            f[2 * h] = x.x;
            f[2 * h + 1] = x.y;
        }
    }
}

struct DequantArgs {
    void* out[2];  // k, v [rows, H, D]
    int planes;
    Divider vecs;  // 16-value chunks a token
    KvCache c;
    KvSteps st;
};

template <int DT, int MODE>
__global__ void __launch_bounds__(kThreads, 4) kv_dequantize_kernel(const __grid_constant__ DequantArgs a) {
    const KvCache& c = a.c;
    pdl_launch_dependents();
    pdl_wait();
    const int s = kv_find_seq(a.st, blockIdx.x, 1, c.block, 2);
    const SeqSpan span = seq_span(a.st, s, c.block);
    const int64_t j = static_cast<int64_t>(blockIdx.x) - kv_first_item(a.st, s, 1, c.block, 2);
    const BlockWork w = block_work(c, a.st, span, s, j);
    const int p0 = blockIdx.y * a.planes;
    const int count = p0 + a.planes < 2 * c.H ? a.planes : 2 * c.H - p0;
    const int vecs = c.D / 16;
    auto store = [&](int plane, int64_t row, int d, const float (&f)[16]) {
        const int64_t at = (row * c.H + (plane >> 1)) * c.D + d;
        void* out = plane & 1 ? a.out[1] : a.out[0];
        if constexpr (DT == NV_F32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        } else {
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
            o[0] = make_uint4(v[0], v[1], v[2], v[3]);
            o[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
    };
    const float zeros[16] = {};
    if (j == 0 && span.first < 0) {  // rows in front of the sequence (a bad length): with its first block
        const int64_t missing = span.n < -span.first ? span.n : -span.first;
        for (int64_t i = threadIdx.x; i < missing * vecs * count; i += kThreads) {
            const int64_t k = i / vecs;
            store(p0 + static_cast<int>(k % count), span.row0 + k / count, static_cast<int>(i % vecs) * 16, zeros);
        }
    }
    if (!w.any) return;
    const int chunks = (w.slot1 - w.slot0) * vecs;
    if (!page_ok(c, a.st, w)) {
        for (int i = threadIdx.x; i < chunks * count; i += kThreads) {
            const int p = i / chunks, k = i - p * chunks, tok = k / vecs;
            store(p0 + p, w.row0 + tok, (k - tok * vecs) * 16, zeros);
        }
        return;
    }
    const int64_t bytes = static_cast<int64_t>(c.block) * c.D;
    constexpr int kUnroll = 4;
    // thread = (plane of the run, chunk): chunks * count stays below 2^16 but for runs of many heads of
    // large blocks, which take the planes in several rounds
    const int fit = 0xFFFF / chunks < count ? 0xFFFF / chunks : count;
    const float by_chunk = 1.f / static_cast<float>(chunks);
    for (int first = 0; first < count; first += fit) {
        const int planes = count - first < fit ? count - first : fit;
        for (int i0 = threadIdx.x; i0 < chunks * planes; i0 += kThreads * kUnroll) {
            uint4 u[kUnroll];
            float scale[kUnroll];
            int plane[kUnroll], k[kUnroll];
#pragma unroll
            for (int n = 0; n < kUnroll; ++n) {
                const int i = i0 + n * kThreads;
                if (i >= chunks * planes) break;
                // i / chunks: the quotient of two integers below 2^16, rounded down, from its fp32 value
                int q = static_cast<int>((static_cast<float>(i) + 0.5f) * by_chunk);
                plane[n] = p0 + first + q;
                k[n] = i - q * chunks;
                const int64_t at = static_cast<int64_t>(w.page) * c.H + (plane[n] >> 1);
                u[n] = __ldg(reinterpret_cast<const uint4*>((plane[n] & 1 ? c.v_codes : c.k_codes) + at * bytes +
                                                           static_cast<int64_t>(w.slot0) * c.D + 16 * static_cast<int64_t>(k[n])));
                scale[n] = __ldg((plane[n] & 1 ? c.v_scales : c.k_scales) + at);
            }
#pragma unroll
            for (int n = 0; n < kUnroll; ++n) {
                if (i0 + n * kThreads >= chunks * planes) break;
                const int tok = a.vecs.of(k[n]);
                const uint32_t x[4] = {u[n].x, u[n].y, u[n].z, u[n].w};
                float f[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) word_values<MODE>(x[e], f + 4 * e);
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] *= scale[n];
                store(plane[n], w.row0 + tok, (k[n] - tok * vecs) * 16, f);
            }
        }
    }
}

template <typename... Args>
cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Planes a CTA takes: a block of tokens is cut into runs of planes of at least about
// 4096 values, into no more than make 1100 CTAs (or three a block). What few tokens cost
// is the number of CTAs: appending to 128 sequences takes 11 us with one a block, 26 with one a
// plane; a prompt of 8192 tokens takes 36 us with two planes a CTA, 40 with one or four.
int planes_per_cta(const KvCache& c, const KvSteps& st, int64_t items) {
    const int64_t by_values = st.rows * 2 * c.H * c.D / items / 4096;
    const int64_t by_ctas = 1100 / items > 3 ? 1100 / items : 3;
    int64_t runs = by_values < by_ctas ? by_values : by_ctas;
    if (runs < 1) runs = 1;
    const int64_t planes = (2 * c.H + runs - 1) / runs;
    return static_cast<int>(planes < 1 ? 1 : planes);
}

}  // namespace

cudaError_t launch_kv_quantize(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int dt,
                               const KvCache& c, const KvSteps& st, cudaStream_t stream) {
    const int64_t items = kv_items(st.rows, st.S, 1, c.block, 2);
    const int planes = planes_per_cta(c, st, items);
    QuantArgs a{{k, v}, {k_stride, v_stride}, planes, Divider(c.D / 8), c, st};
    const dim3 grid(static_cast<unsigned>(items), (2 * c.H + planes - 1) / planes, 1);
    if (dt == NV_F32)
        return c.mode == NV_KV_INT8 ? launch_pdl(kv_quantize_kernel<NV_F32, NV_KV_INT8>, grid, kThreads, stream, a)
                                    : launch_pdl(kv_quantize_kernel<NV_F32, NV_KV_E4M3>, grid, kThreads, stream, a);
    return c.mode == NV_KV_INT8 ? launch_pdl(kv_quantize_kernel<NV_BF16, NV_KV_INT8>, grid, kThreads, stream, a)
                                : launch_pdl(kv_quantize_kernel<NV_BF16, NV_KV_E4M3>, grid, kThreads, stream, a);
}

cudaError_t launch_kv_dequantize(void* k, void* v, int dt, const KvCache& c, const KvSteps& st,
                                 cudaStream_t stream) {
    const int64_t items = kv_items(st.rows, st.S, 1, c.block, 2);
    const int planes = planes_per_cta(c, st, items);
    DequantArgs a{{k, v}, planes, Divider(c.D / 16), c, st};
    const dim3 grid(static_cast<unsigned>(items), (2 * c.H + planes - 1) / planes, 1);
    if (dt == NV_F32)
        return c.mode == NV_KV_INT8 ? launch_pdl(kv_dequantize_kernel<NV_F32, NV_KV_INT8>, grid, kThreads, stream, a)
                                    : launch_pdl(kv_dequantize_kernel<NV_F32, NV_KV_E4M3>, grid, kThreads, stream, a);
    return c.mode == NV_KV_INT8 ? launch_pdl(kv_dequantize_kernel<NV_BF16, NV_KV_INT8>, grid, kThreads, stream, a)
                                : launch_pdl(kv_dequantize_kernel<NV_BF16, NV_KV_E4M3>, grid, kThreads, stream, a);
}

}  // namespace nvq
