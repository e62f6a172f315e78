// Attention over the paged 8-bit cache for many query rows a sequence (bf16, 64 or
// 128 values a head), on the tensor cores (tcgen05).
//
// An item is 256 query rows of one sequence and key/value head (row = (token,
// query head of the group)) against its visible tokens, 128 at a time. One CTA per
// SM and item; rows form two subtiles of 128 that share every converted key and
// value tile and take turns on the tensor core: while one subtile's softmax runs, the
// other's products do. An item of at most 128 rows (a few tokens of many heads, a prompt's
// end) is one subtile: both softmax groups hold it, each takes every other tile of
// tokens, and they join at the end (64 sequences of 8192, 20 rows a head: 700 us with the
// second group idle, 440 so; as two tiles of the kernel for few rows, 710).
//   warp 0           issues the products: S = Q K^T (K-major operands), O += P V
//                    with P from TMEM and V read along tokens (MN-major), so V
//                    needs no transpose
//   warp 1           looks pages and scales up, four tiles at a time, up to eight ahead, and
//                    asks the L2 for their codes
//   warps 4-7, 8-11  softmax of subtile 0, 1: thread = row = TMEM lane; scores
//                    arrive in TMEM, weights go back over them as fp16
//   warps 12-15      converters: 8-bit codes from global memory (a tile of them in
//                    flight in registers), exact fp16 into swizzled shared tiles
//                    [token][value], a ring of two K and two V tiles
// Sixteen warps leave 128 registers a thread and none spills: with 200 KB of shared memory taken there
// is next to no L1, and spilled registers would come back from the L2.
// TMEM (512 columns): S0, S1 (128 each, P over the first 64), O0, O1 (D each).
//
// Block scales never touch the tiles: keys' are factors of the scores, values' join
// the exponent (weights are 2^(z + lg)), and the weights' sum takes them out again.
// An item whose value scales are too far apart for that (2^24; blocks of zeros do not count) goes row by
// row in fp32: a prompt of 8192 with one such block takes 70 ms if it is the last, 250 if the first.
// A row's reference follows its running maximum only when that passes it by
// kSlack, so rescaling O in TMEM is rare and the softmax warps do it themselves.
//
// Bound: neither the tensor core (38 % busy) nor the exponential unit (39 %), but the chain of
// one subtile's step, about 4600 cycles for a pair of tiles: its own products (825; the other subtile's
// run under its softmax), then a softmax of 2900, whose 128 exponentials a thread issue one in 8 cycles
// at best (1024 of them) and in 12.7 as one warp a scheduler reaches; some 900 cycles between them are
// not accounted for. Measured at a prompt
// of 8192 (32 heads over 8, D = 128), each slower than the 665 to 683 us (827 to 805 TFLOP/s, from GPU to GPU) of this
// form: scores held in registers through an unrolled loop, four softmax warpgroups with two threads a row (745), an issuing warp a
// subtile, a share of the exponentials as polynomials on the FMA pipe.
#include <cstdint>

#include "kv_mma.cuh"
#include "kv_plain.cuh"

namespace nvq {
namespace {

constexpr int kRows = 256;     // rows an item
constexpr int kTile = 128;     // tokens a tile
constexpr int kIssueWarp = 0, kLookupWarp = 1, kSoftmaxWarp0 = 4, kSoftmaxWarps = 8, kConvertWarp0 = 12, kConvertWarps = 4;
constexpr int kThreads = 32 * 16;
constexpr int kTmemCols = 512;
constexpr int kMeta = 8;       // ring of per-tile lookups
constexpr int kMetaBatch = 4;  // tiles looked up at once
constexpr int kChunks = kTile / 16;

struct PrefillArgs {
    KvAttn a;
    KvCache c;
    KvSteps st;
    int64_t items;    // row tiles of all sequences, at most
    int splits;       // parts the tokens of an item are cut into
    int row_min;      // sequences of at most this many flattened rows are another kernel's
    float* part_o;    // [rows * Hq][splits][D]
    float* part_lse;  // [rows * Hq][splits]
};

struct ChunkScales {  // of 16 tokens
    float ks;   // negative: not seen
    float lg, inv;
    float pad;
};

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
// The loads before it are complete; tied to the registers so that no use moves ahead of it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
// No wait (tc::tmem_st_wait), and no claim on other memory: loads may move across.
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// fp16 operands, fp32 accumulator; b_mn: B is read along N (MN-major).
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}
// The products and commits of the issuing warp: all lanes go along (uniform addresses stay
// in uniform registers), one elected lane issues.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
// MN-major, 128-byte swizzle: rows of 64 values; 8-token groups 1024 bytes apart
// (stride offset), the next 64 values `lead` bytes on (leading offset).
__device__ __forceinline__ uint64_t sw128_mn_desc(const void* p, uint32_t lead) {
    const uint64_t addr = smem_u32(p);
    return ((addr & 0x3FFFFull) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Byte offset of 16-byte piece `piece` (8 values) of row r in a [rows][64 values] swizzled tile.
__device__ __forceinline__ uint32_t sw128_at(int r, int piece) {
    return static_cast<uint32_t>((r >> 3) * 1024 + (r & 7) * 128 + ((piece ^ (r & 7)) << 4));
}

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// What a 16-token chunk's scores are multiplied by: positive even where keys or
// queries are all zero, so that a score of -infinity (not seen) stays one.
__device__ __forceinline__ float score_factor(float zc, float ks) { return fmaxf(zc * ks, 1e-37f); }

// The rows of a wide item (value scales too far apart for fp16 weights), every fourth by each 128 threads.
template <int MODE, int D>
__device__ __noinline__ void wide_item(const PrefillArgs& p, const SeqSpan span, int s, int h, int f0, int rows, int lo, int hi,
                                       PlainScratch<D>* scratch) {
    constexpr int kTeams = kThreads / kPlainThreads;
    const int G = p.a.Hq / p.c.H, team = threadIdx.x / kPlainThreads, d = threadIdx.x % kPlainThreads;
    for (int row = team; row < rows; row += kTeams) {
        const int f = f0 + row, hq = h * G + f % G;
        const int64_t t = span.row0 + f / G, at = t * p.a.Hq + hq;
        const PlainRow r = plain_row<NV_BF16, MODE>(p.a, p.c, p.st, s, span, t, hq, lo, hi, d, scratch[team], [team] {
            asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kPlainThreads) : "memory");
        });
        if (p.splits > 1) {
            const int64_t part = at * p.splits + blockIdx.y;
            if (d < D) p.part_o[part * D + d] = r.out[0];
            if (d == 0) p.part_lse[part] = r.l != r.l ? 0.f : r.l > 0.f ? r.m * kLog2e + log2f(r.l) : -INFINITY;
        } else if (d < D) {
            static_cast<uint16_t*>(p.a.out)[at * D + d] = f32_to_bf16_bits(r.out[0]);
        }
    }
}

template <int D>
struct Smem {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalf = 128 * 128;               // bytes of 128 rows x 64 values
    static constexpr int kSub = kHalves * kHalf;          // a Q subtile, a K or V tile
    static constexpr int kSlots = 4;                      // K, V, K, V
    static constexpr int kBytes = (2 + kSlots) * kSub + 1024;
};

template <int MODE, int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_prefill_kernel(const __grid_constant__ PrefillArgs p) {
    using L = Smem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* q_smem = smem;                      // [2][kSub]
    uint8_t* ring = smem + 2 * L::kSub;          // [4][kSub]
    __shared__ __align__(8) uint64_t full[4], empty[4], q_full[2], s_full[2], p_full[2], o_full[2],
        m_full[kMeta], m_empty[kMeta];
    __shared__ ChunkScales scales[kMeta][kChunks];
    __shared__ int64_t places[kMeta][kChunks];  // byte offset of the chunk's codes of this head, -1: none
    __shared__ uint32_t tmem_slot, vmax_bits, vmin_bits;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    pdl_launch_dependents();
    pdl_wait();

    // ---- the item: later rows first, they see the most tokens
    const int G = p.a.Hq / p.c.H;
    const int h = blockIdx.x % p.c.H;
    const int64_t item = p.items - 1 - blockIdx.x / p.c.H;
    const int s = kv_find_seq(p.st, item, G, kRows, 1);
    const SeqSpan span = seq_span(p.st, s, p.c.block);
    const int64_t j_item = item - kv_first_item(p.st, s, G, kRows, 1);
    const int64_t seq_rows = static_cast<int64_t>(span.n) * G;
    if (j_item < 0 || j_item * kRows >= seq_rows || seq_rows <= p.row_min) return;
    const int f0 = static_cast<int>(j_item * kRows);
    const int rows = seq_rows - f0 < kRows ? static_cast<int>(seq_rows - f0) : kRows;
    // One subtile of rows: both softmax groups take it, each every other tile of tokens, and join at the end.
    const bool alternate = rows <= kRows / 2;
    const int turns = alternate ? 2 : 1;  // tiles from one of a group's to its next
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&full[i], kConvertWarps);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 128);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
        }
        for (int i = 0; i < kMeta; ++i) {
            mbar_init(&m_full[i], 1);
            mbar_init(&m_empty[i], (alternate ? kSoftmaxWarps / 2 : kSoftmaxWarps) + kConvertWarps);
        }
        mbar_init_fence();
        vmax_bits = 0;
        vmin_bits = 0x7F800000u;
    }
    int lo = 0, hi = span.len;
    if (p.a.causal) {
        const int p0 = span.first + f0 / G, p1 = span.first + (f0 + rows - 1) / G;
        hi = p1 + 1 < hi ? p1 + 1 : hi;
        if (p.a.window > 0 && p0 + 1 > p.a.window) lo = p0 + 1 - p.a.window;
    }
    const int lo_seen = lo;  // what is in front of it only shares a tile with what the window shows
    lo = lo / kTile * kTile;
    int tiles = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
    if (p.splits > 1) {
        const int per = (tiles + p.splits - 1) / p.splits;
        const int z = blockIdx.y;
        lo += z * per * kTile;
        tiles = tiles - z * per < per ? tiles - z * per : per;
        if (tiles < 0) tiles = 0;
        if (lo + tiles * kTile < hi) hi = lo + tiles * kTile;
    }

    // ---- the largest value scale of the item: weights carry value scales relative to it (and the smallest but zero)
    if (tiles > 0) {
        const int b0 = (lo > lo_seen ? lo : lo_seen) / p.c.block, b1 = (hi - 1) / p.c.block;
        float most = 0.f, least = INFINITY;
        for (int b = b0 + tid; b <= b1; b += kThreads) {
            const int32_t page = __ldg(p.st.pages + static_cast<int64_t>(s) * p.st.max_pages + b);
            if (page >= 0 && page < p.c.P) {
                const float vs = __ldg(p.c.v_scales + static_cast<int64_t>(page) * p.c.H + h);
                most = fmaxf(most, vs);
                if (vs > 0.f) least = fminf(least, vs);
            }
        }
        __syncthreads();  // vmax_bits and vmin_bits initialised
        const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
        const uint32_t low_bits = __reduce_min_sync(0xffffffffu, __float_as_uint(least));
        if (lane == 0 && bits) {
            atomicMax(&vmax_bits, bits);
            atomicMin(&vmin_bits, low_bits);
        }
    }
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const float vmax = __uint_as_float(vmax_bits);
    bool ok = true;

    if (vmax > 0.f && log2f(__uint_as_float(vmin_bits)) - log2f(vmax) < kLgWide) {
        wide_item<MODE, D>(p, span, s, h, f0, rows, lo, hi, reinterpret_cast<PlainScratch<D>*>(q_smem));
    } else if (warp >= kSoftmaxWarp0 && warp < kSoftmaxWarp0 + kSoftmaxWarps) {
        // ------------------------------------------------------------- softmax
        const int sub = (warp - kSoftmaxWarp0) >> 2;
        const int r_sub = tid & 127;              // row of the subtile = TMEM lane
        const int row = alternate ? r_sub : sub * 128 + r_sub;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + static_cast<uint32_t>(sub * 128);
        const uint32_t o_at = tmem + lanes + 256u + static_cast<uint32_t>(sub * D);
        const int f = f0 + row, tok = f / G;
        int row_lo = 0, row_hi = span.len;
        float zc = 0.f;
        bool bad = false;
        int64_t out_row = 0;
        {
            const uint4* q = nullptr;
            if (row < rows) {
                const int pos = span.first + tok;
                if (p.a.causal) {
                    row_hi = pos + 1 < span.len ? pos + 1 : span.len;
                    if (p.a.window > 0 && pos + 1 > p.a.window) row_lo = pos + 1 - p.a.window;
                }
                const int hq = h * G + f % G;
                out_row = (span.row0 + tok) * p.a.Hq + hq;
                q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.a.q) +
                                                   (span.row0 + tok) * p.a.q_stride + static_cast<int64_t>(hq) * D);
            }
            uint32_t most = 0;
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) {
                const uint4 r = q ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) most = max(most, max((u[j] << 16) & 0x7FFFFFFFu, u[j] & 0x7FFF0000u));
            }
            bad = most >= 0x7F800000u;
            const uint32_t ex = row_exponent(most);
            // a negative scale goes into the queries: scores times zc keep their order
            const float down = p.a.scale < 0.f ? -pow2_bits(254u - ex) : pow2_bits(254u - ex);
            zc = fabsf(p.a.scale) * kLog2e * pow2_bits(ex);
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) {  // the second time from the L1
                const uint4 r = q ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {r.x, r.y, r.z, r.w};
                uint32_t x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[j] = f2_to_h2(__uint_as_float(u[j] << 16) * down, __uint_as_float(u[j] & 0xFFFF0000u) * down);
                *reinterpret_cast<uint4*>(q_smem + sub * L::kSub + (i >> 3) * L::kHalf + sw128_at(r_sub, i & 7)) =
                    make_uint4(x[0], x[1], x[2], x[3]);
            }
            fence_proxy_async();
            mbar_arrive(&q_full[sub]);
        }
        float ref = -INFINITY, l = 0.f;
        const int first = alternate ? sub : 0;
        for (int i = first, n = 0; ok && i < tiles; i += turns, ++n) {
            const int j0 = lo + i * kTile;
            const int ms = i & (kMeta - 1);
            ok = mbar_wait(&m_full[ms], (i / kMeta) & 1, 0x71) && mbar_wait(&s_full[sub], n & 1, 0x72);
            if (!ok) break;
            tc::tc_fence_after();
            const ChunkScales* ts = scales[ms];
            // does every row of the warp see all of the tile? If not, the scores that are not seen become
            // -infinity in place, so that the two passes need not ask
            bool all = row_lo <= j0 && row_hi >= j0 + kTile;
            all &= ts[lane & (kChunks - 1)].ks >= 0.f;
            if (!__all_sync(0xffffffffu, all)) {
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    uint32_t v[16];
                    tmem_ld_x16(s_at + 16u * c, v);
                    tmem_ld_wait(v);
                    const int from = ts[c].ks >= 0.f ? row_lo - j0 - 16 * c : 16, to = row_hi - j0 - 16 * c;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (e < from || e >= to) v[e] = 0xFF800000u;
                    tc::tmem_st_x16_async(s_at + 16u * c, v);
                }
                tc::tmem_st_wait();
            }
            // Scores are read twice, 16 at a time with the next 16 in flight, in rolled loops: the code of
            // the three roles has to stay in the instruction caches (unrolled, the warps waited for
            // instructions more than for anything else).
            uint32_t sv[2][16];
            tmem_ld_x16(s_at, sv[0]);
            float mx = -INFINITY;
            auto largest = [&](const uint32_t (&v)[16], const ChunkScales& t) {
                float m0 = __uint_as_float(v[0]), m1 = __uint_as_float(v[1]);
#pragma unroll
                for (int e = 2; e < 14; e += 4) {
                    m0 = max3(m0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                    m1 = max3(m1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                }
                mx = fmaxf(mx, fmaf(max3(fmaxf(m0, m1), __uint_as_float(v[14]), __uint_as_float(v[15])), score_factor(zc, t.ks), t.lg));
            };
#pragma unroll 1
            for (int c = 0; c < kChunks; c += 2) {
                const ChunkScales ta = ts[c], tb = ts[c + 1];
                tmem_ld_wait(sv[0]);
                tmem_ld_x16(s_at + 16u * (c + 1), sv[1]);
                largest(sv[0], ta);
                tmem_ld_wait(sv[1]);
                tmem_ld_x16(s_at + 16u * ((c + 2) & (kChunks - 1)), sv[0]);  // behind the last: the first again
                largest(sv[1], tb);
            }
            const bool up = mx > ref + kSlack;
            if (__any_sync(0xffffffffu, up)) {
                // each row by itself; the previous tile's P V is complete (its commit came before this S)
                const float fct = up ? exp2f(ref - mx) : 1.f;
                ref = up ? mx : ref;
                l *= fct;
                if (n > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t ov[16];
                        tmem_ld_x16(o_at + 16u * c, ov);
                        tmem_ld_wait(ov);
#pragma unroll
                        for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * fct);
                        tc::tmem_st_x16_async(o_at + 16u * c, ov);
                    }
                    tc::tmem_st_wait();
                }
            }
            const float minus_ref = kLift - (ref > -INFINITY ? ref : 0.f);
            // a chunk's weights, as fp16 over scores that are done
            auto weigh = [&](const uint32_t (&v)[16], const ChunkScales& t, int c) {
                uint32_t pw[8];
                uint64_t sum[2] = {};
                const uint32_t k1 = __float_as_uint(score_factor(zc, t.ks)), b1 = __float_as_uint(t.lg + minus_ref);
                const uint64_t k2 = tc::f2_pack(k1, k1), b2 = tc::f2_pack(b1, b1);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const uint64_t z = tc::f2_fma(tc::f2_pack(v[e], v[e + 1]), k2, b2);
                    const float w0 = exp2_approx(__uint_as_float(static_cast<uint32_t>(z)));
                    const float w1 = exp2_approx(__uint_as_float(static_cast<uint32_t>(z >> 32)));
                    sum[e / 2 & 1] = f2_add(sum[e / 2 & 1], tc::f2_pack(__float_as_uint(w0), __float_as_uint(w1)));
                    pw[e / 2] = f2_to_h2(w0, w1);
                }
                tmem_st_x8(s_at + 8u * c, pw);
                sum[0] = f2_add(sum[0], sum[1]);
                l = fmaf(__uint_as_float(static_cast<uint32_t>(sum[0])) + __uint_as_float(static_cast<uint32_t>(sum[0] >> 32)), t.inv, l);
            };
            ChunkScales ta = ts[0], tb = ts[1];
#pragma unroll 1
            for (int c = 0; c < kChunks; c += 2) {
                const int next = (c + 2) & (kChunks - 1);
                tmem_ld_wait(sv[0]);
                tmem_ld_x16(s_at + 16u * (c + 1), sv[1]);
                weigh(sv[0], ta, c);
                ta = ts[next];
                tmem_ld_wait(sv[1]);
                tmem_ld_x16(s_at + 16u * next, sv[0]);  // behind the last: nobody's
                weigh(sv[1], tb, c + 1);
                tb = ts[next + 1];
            }
            tmem_ld_wait(sv[0]);
            tc::tmem_st_wait();
            tc::tc_fence_before();
            mbar_arrive(&p_full[sub]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&m_empty[ms]);
        }
        // ---- output
        const bool has_o = first < tiles;
        if (ok && has_o) ok = mbar_wait(&o_full[sub], 0, 0x73);
        tc::tc_fence_after();
        float4* other = reinterpret_cast<float4*>(ring);  // [D / 4][128]: what the second group found, then its reference and sum
        float f_own = 1.f, f_other = 0.f;
        if (alternate && tiles > 1) {
            float2* other_sums = reinterpret_cast<float2*>(other + 128 * (D / 4));
            if (sub == 1) {
                // the products are done with the tiles that this goes over
                if (ok) ok = mbar_wait(&o_full[0], 0, 0x7E);
                if (ok) {
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t ov[16];
                        tmem_ld_x16(o_at + 16u * c, ov);
                        tmem_ld_wait(ov);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            other[(4 * c + e) * 128 + r_sub] = make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                                                                           __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
                    }
                    other_sums[r_sub] = make_float2(ref, l);
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (sub == 0) {
                const float2 o = other_sums[r_sub];
                const float top = fmaxf(ref, o.x);
                f_own = ref > -INFINITY ? exp2f(ref - top) : 0.f;
                f_other = o.x > -INFINITY ? exp2f(o.x - top) : 0.f;
                ref = top;
                l = l * f_own + o.y * f_other;
            }
        }
        if (ok && (sub == 0 || !alternate)) {
            const bool live = row < rows;
            const float inv = bad ? NAN : ref > -INFINITY ? vmax / l : 0.f;  // no reference: nothing was seen
            const int64_t at = p.splits > 1 ? out_row * p.splits + blockIdx.y : 0;
#pragma unroll 2
            for (int c = 0; c < D / 16; ++c) {
                uint32_t ov[16];
                if (has_o) {
                    tmem_ld_x16(o_at + 16u * c, ov);
                    tmem_ld_wait(ov);
                    if (alternate && tiles > 1) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float y = reinterpret_cast<const float*>(other + (4 * c + e / 4) * 128 + r_sub)[e & 3];
                            ov[e] = __float_as_uint(fmaf(__uint_as_float(ov[e]), f_own, y * f_other));
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) ov[e] = 0;
                }
                if (!live) continue;
                if (p.splits > 1) {
                    float4* o = reinterpret_cast<float4*>(p.part_o + at * D + 16 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = make_float4(__uint_as_float(ov[4 * e]) * inv, __uint_as_float(ov[4 * e + 1]) * inv,
                                           __uint_as_float(ov[4 * e + 2]) * inv, __uint_as_float(ov[4 * e + 3]) * inv);
                } else {
                    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + out_row * D + 16 * c);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t x[4];
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            x[n] = tc::f2_to_bf2(__uint_as_float(ov[8 * e + 2 * n]) * inv, __uint_as_float(ov[8 * e + 2 * n + 1]) * inv);
                        o[e] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
            }
            if (live && p.splits > 1)
                p.part_lse[at] = bad ? 0.f : ref > -INFINITY ? ref - kLift + log2f(l) : -INFINITY;
        }
        tc::tc_fence_before();
    } else if (warp >= kConvertWarp0) {
        // ---------------------------------------------------------- converters
        const int ct = tid - 32 * kConvertWarp0;
        // A thread takes 16 values (16 bytes of codes, two 16-byte pieces of fp16) of every 16th (32nd) token.
        // Eight neighbours are two tokens by four such runs of one half of 64 values, whose pieces
        // fall into different banks; a warp reads whole rows of codes.
        constexpr int kStep = D == 128 ? 16 : 32;      // tokens a pass of all threads
        constexpr int kPasses = kTile / 2 / kStep;     // passes of half a tile: 4 (D 128) or 2 (D 64)
        const int run = lane & 3, half = D == 128 ? lane >> 3 & 1 : 0;
        const int tok0 = D == 128 ? (ct >> 5) * 4 + (lane >> 4) * 2 + (lane >> 2 & 1) : ct >> 2;
        const uint32_t at0 = half * L::kHalf + sw128_at(tok0, 2 * run), at1 = half * L::kHalf + sw128_at(tok0, 2 * run + 1);
        const uint32_t code0 = (tok0 & 15) * D + 64 * half + 16 * run;
        // codes of tokens 64 part .. of tile i
        auto load = [&](const uint8_t* codes, int i, int part, uint4 (&raw)[kPasses]) {
            const int64_t* at = places[i & (kMeta - 1)] + 4 * part + (tok0 >> 4);
            const int left = hi - (lo + i * kTile) - 64 * part - tok0;
#pragma unroll
            for (int n = 0; n < kPasses; ++n) {
                const int64_t o = at[n * (kStep / 16)];
                raw[n] = make_uint4(0, 0, 0, 0);
                if (o >= 0 && kStep * n < left) raw[n] = __ldg(reinterpret_cast<const uint4*>(codes + o + code0));
            }
        };
        auto convert = [&](const uint4 (&raw)[kPasses], uint8_t* tile, int part) {
            uint8_t* t0 = tile + at0 + part * (64 * 128);
            uint8_t* t1 = tile + at1 + part * (64 * 128);
#pragma unroll
            for (int n = 0; n < kPasses; ++n) {
                const uint32_t a = prepare_word<MODE>(raw[n].x), b = prepare_word<MODE>(raw[n].y);
                const uint32_t c = prepare_word<MODE>(raw[n].z), d = prepare_word<MODE>(raw[n].w);
                *reinterpret_cast<uint4*>(t0 + n * (kStep * 128)) =
                    make_uint4(pair_lo_h2<MODE>(a), pair_hi_h2<MODE>(a), pair_lo_h2<MODE>(b), pair_hi_h2<MODE>(b));
                *reinterpret_cast<uint4*>(t1 + n * (kStep * 128)) =
                    make_uint4(pair_lo_h2<MODE>(c), pair_hi_h2<MODE>(c), pair_lo_h2<MODE>(d), pair_hi_h2<MODE>(d));
            }
        };
        auto done = [&](uint64_t* bar) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // Halves of K, then of V; a half's registers take the next tile's codes when they are converted, so that
        // a whole tile's are in flight or waiting. One subtile of rows waits for the codes: it asks as early
        // as it can. Two wait for their softmax: the loads stand behind the fence that publishes a tile, which
        // would wait for them (prompt of 8192: 668 us, 681 with the early loads; 20 rows: 470 and 440).
        uint4 k0[kPasses], k1[kPasses], v0[kPasses], v1[kPasses];
        auto next = [&](const uint8_t* codes, int i, int part, uint4 (&raw)[kPasses]) {
            if (i < tiles) load(codes, i, part, raw);
        };
        auto looked_up = [&](int i) {  // tile i's places have been read
            __syncwarp();
            if (lane == 0 && i < tiles) mbar_arrive(&m_empty[i & (kMeta - 1)]);
        };
        if (tiles > 0) ok = mbar_wait(&m_full[0], 0, 0x74);
        if (ok) {
            next(p.c.k_codes, 0, 0, k0);
            next(p.c.k_codes, 0, 1, k1);
            next(p.c.v_codes, 0, 0, v0);
            next(p.c.v_codes, 0, 1, v1);
            looked_up(0);
        }
        for (int i = 0; ok && i < tiles; ++i) {
            const int ks = 2 * (i & 1), vs = ks + 1;
            const uint32_t free_parity = ((i >> 1) & 1) ^ 1;
            ok = mbar_wait(&empty[ks], free_parity, 0x75);
            if (ok && i + 1 < tiles) ok = mbar_wait(&m_full[(i + 1) & (kMeta - 1)], ((i + 1) / kMeta) & 1, 0x7B);
            if (!ok) break;
            convert(k0, ring + ks * L::kSub, 0);
            if (alternate) next(p.c.k_codes, i + 1, 0, k0);
            convert(k1, ring + ks * L::kSub, 1);
            if (alternate) next(p.c.k_codes, i + 1, 1, k1);
            done(&full[ks]);
            if (!alternate) {
                next(p.c.k_codes, i + 1, 0, k0);
                next(p.c.k_codes, i + 1, 1, k1);
            }
            ok = mbar_wait(&empty[vs], free_parity, 0x7C);
            if (!ok) break;
            convert(v0, ring + vs * L::kSub, 0);
            if (alternate) next(p.c.v_codes, i + 1, 0, v0);
            convert(v1, ring + vs * L::kSub, 1);
            if (alternate) next(p.c.v_codes, i + 1, 1, v1);
            done(&full[vs]);
            if (!alternate) {
                next(p.c.v_codes, i + 1, 0, v0);
                next(p.c.v_codes, i + 1, 1, v1);
            }
            looked_up(i + 1);
        }
    } else {
      if (warp == kLookupWarp) {
        // ------------------------------------------------- pages and scales: lane = (tile of four, chunk of 16 tokens)
        const float lg_max = log2f(vmax);
        for (int i0 = 0; ok && i0 < tiles; i0 += kMetaBatch) {
            const int i = i0 + lane / kChunks, c = lane % kChunks;
            const int j = lo + i * kTile + 16 * c;
            ChunkScales t{-1.f, 0.f, 1.f, 0.f};
            int64_t at = -1;
            if (i < tiles && j < hi && j + 16 > lo_seen) {
                const int b = j / p.c.block;
                const int page = page_of(p.st, p.c, s, b);
                if (page >= 0) {
                    const int64_t ph = static_cast<int64_t>(page) * p.c.H + h;
                    const float vs = __ldg(p.c.v_scales + ph);
                    at = (ph * p.c.block + (j - b * p.c.block)) * D;
                    t.ks = __ldg(p.c.k_scales + ph);
                    t.lg = vs > 0.f ? log2f(vs) - lg_max : kLgZero;
                    t.inv = exp2f(-t.lg);
                    prefetch_l2(p.c.k_codes + at, 16 * D);
                    prefetch_l2(p.c.v_codes + at, 16 * D);
                }
            }
            for (int n = i0; ok && n < i0 + kMetaBatch && n < tiles; ++n)
                ok = mbar_wait(&m_empty[n & (kMeta - 1)], ((n / kMeta) & 1) ^ 1, 0x7D);
            if (!ok) break;
            if (i < tiles) {
                scales[i & (kMeta - 1)][c] = t;
                places[i & (kMeta - 1)][c] = at;
            }
            __syncwarp();
            if (i < tiles && c == 0) mbar_arrive(&m_full[i & (kMeta - 1)]);
        }
      } else if (warp == kIssueWarp) {
        if (tiles > 0) {
            // ------------------------------------------------------ the products
            constexpr uint32_t idesc_s = idesc_f16(128, kTile, 0), idesc_o = idesc_f16(128, D, 1);
            // everything but the tile's ring slot (kSub apart) is fixed
            const uint64_t q_desc = tc::sw128_desc(q_smem), k_desc = tc::sw128_desc(ring);
            const uint64_t v_desc = sw128_mn_desc(ring + L::kSub, L::kHalf);
            constexpr uint64_t kSubUnits = L::kSub >> 4;
            auto qk = [&](int sub, int i) {
                const uint64_t a = q_desc + (sub ? kSubUnits : 0), b = k_desc + (i & 1 ? 2 * kSubUnits : 0);
                const uint32_t d = tmem + sub * 128;
#pragma unroll 2
                for (int k = 0; k < D / 16; ++k) {
                    constexpr uint64_t kHalfUnits = L::kHalf >> 4;
                    const uint64_t off = (k >> 2) * kHalfUnits + (k & 3) * 2;
                    mma_ss(d, a + off, b + off, idesc_s, k > 0);
                }
            };
            auto pv = [&](int sub, int i, bool add) {
                const uint64_t b = v_desc + (i & 1 ? 2 * kSubUnits : 0);
                const uint32_t d = tmem + 256 + sub * D, a = tmem + sub * 128;
#pragma unroll 2
                for (int k = 0; k < kTile / 16; ++k) mma_ts(d, a + 8 * k, b + k * 128, idesc_o, add || k > 0);
            };
            // the first products, then each softmax group's next as its weights arrive. K's and V's tiles are in
            // slots by their number's parity, freed when every group that reads them has its products.
            if (alternate) {
                for (int i = 0; ok && i < 2 && i < tiles; ++i) {
                    ok = mbar_wait(&full[2 * i], 0, 0x76) && mbar_wait(&q_full[i], 0, 0x77);
                    if (!ok) break;
                    tc::tc_fence_after();
                    qk(i, i);
                    commit_elected(&s_full[i]);
                    commit_elected(&empty[2 * i]);
                }
                for (int i = 0; ok && i < tiles; ++i) {
                    const int sub = i & 1, ks = 2 * sub, vs = ks + 1;
                    const uint32_t ph = (i >> 1) & 1;
                    ok = mbar_wait(&p_full[sub], ph, 0x78) && mbar_wait(&full[vs], ph, 0x79);
                    if (!ok) break;
                    tc::tc_fence_after();
                    pv(sub, i, i > 1);
                    commit_elected(&empty[vs]);
                    if (i + 2 >= tiles) {
                        commit_elected(&o_full[sub]);
                        continue;
                    }
                    ok = mbar_wait(&full[ks], ph ^ 1, 0x7A);
                    if (!ok) break;
                    tc::tc_fence_after();
                    qk(sub, i);
                    commit_elected(&s_full[sub]);
                    commit_elected(&empty[ks]);
                }
            } else {
                ok = mbar_wait(&full[0], 0, 0x76);
                for (int sub = 0; ok && sub < 2; ++sub) {
                    ok = mbar_wait(&q_full[sub], 0, 0x77);
                    if (!ok) break;
                    tc::tc_fence_after();
                    qk(sub, 0);
                    commit_elected(&s_full[sub]);
                }
                if (ok) commit_elected(&empty[0]);
                for (int i = 0; ok && i < tiles; ++i) {
                    const uint32_t ph = (i >> 1) & 1, phn = ((i + 1) >> 1) & 1;
                    const int ks = 2 * ((i + 1) & 1), vs = 2 * (i & 1) + 1;
                    for (int sub = 0; ok && sub < 2; ++sub) {
                        ok = mbar_wait(&p_full[sub], i & 1, 0x78) && (sub || mbar_wait(&full[vs], ph, 0x79));
                        if (!ok) break;
                        tc::tc_fence_after();
                        pv(sub, i, i > 0);
                        if (i + 1 == tiles) commit_elected(&o_full[sub]);
                        if (sub) commit_elected(&empty[vs]);
                        if (i + 1 < tiles) {
                            if (!sub) {
                                ok = mbar_wait(&full[ks], phn, 0x7A);
                                if (!ok) break;
                                tc::tc_fence_after();
                            }
                            qk(sub, i + 1);
                            commit_elected(&s_full[sub]);
                            if (sub) commit_elected(&empty[ks]);
                        }
                    }
                }
            }
        }
        __syncwarp();
      }
    }
    __syncthreads();
    if (warp == kIssueWarp) {
        tc::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

// Join the parts of every row: one warp per (row, query head), parts in order.
template <int D>
__global__ void __launch_bounds__(128) kv_attn_prefill_join_kernel(const __grid_constant__ PrefillArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (at >= p.st.rows * p.a.Hq) return;
    const int64_t t = at / p.a.Hq;
    const int s = kv_find_seq(p.st, t, 1, 1, 0);
    const SeqSpan span = seq_span(p.st, s, p.c.block);
    if (t < span.row0 || t >= span.row0 + span.n || static_cast<int64_t>(span.n) * (p.a.Hq / p.c.H) <= p.row_min) return;
    float top = -INFINITY;
    for (int k = lane; k < p.splits; k += 32) top = fmaxf(top, __ldcg(p.part_lse + at * p.splits + k));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == -INFINITY) top = 0.f;
    constexpr int V = D / 32;
    float acc[V] = {}, all = 0.f;
#pragma unroll 4
    for (int k = 0; k < p.splits; ++k) {
        const float e = exp2f(__ldcg(p.part_lse + at * p.splits + k) - top);
        all += e;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(p.part_o + (at * p.splits + k) * D + lane * V + i));
            acc[i] = fmaf(e, x.x, acc[i]);
            acc[i + 1] = fmaf(e, x.y, acc[i + 1]);
        }
    }
    const float inv = all > 0.f ? 1.f / all : 0.f;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.a.out) + at * D + lane * V);
#pragma unroll
    for (int i = 0; i < V; i += 2) out[i / 2] = tc::f2_to_bf2(acc[i] * inv, acc[i + 1] * inv);
}

template <int MODE, int D>
cudaError_t launch(const PrefillArgs& p, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(kv_attn_prefill_kernel<MODE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    // Not launched programmatically: its CTAs take a whole SM each, and early ones only keep the last
    // of the kernel before it from theirs (ragged chunks, behind another kernel: 335 -> 320 us).
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.items * p.c.H), p.splits, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Smem<D>::kBytes;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kv_attn_prefill_kernel<MODE, D>, p);
}
template <int D>
cudaError_t launch_join(const PrefillArgs& p, cudaStream_t stream) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.st.rows * p.a.Hq + 3) / 4), 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_attn_prefill_join_kernel<D>, p);
}
PrefillArgs prefill_args(const KvAttn& a, const KvCache& c, const KvSteps& st, const KvPrefillPlan& plan, int row_min,
                         void* workspace) {
    PrefillArgs p{a, c, st, plan.items, plan.splits, row_min, nullptr, nullptr};
    if (plan.splits > 1) {
        p.part_o = static_cast<float*>(workspace);
        p.part_lse = p.part_o + st.rows * a.Hq * plan.splits * c.D;
    }
    return p;
}

}  // namespace

unsigned int kv_attn_prefill_error_take() { return pipeline_error_take(); }

KvPrefillPlan kv_prefill_plan(const KvPrefillSizes& z, int num_sms) {
    KvPrefillPlan r{};
    r.items = kv_items(z.rows, static_cast<int>(z.S), z.Hq / z.H, kRows, 1);
    // few row tiles: cut the tokens, down to two tiles of them a part
    const int64_t ctas = r.items * z.H;
    const int64_t tiles = (z.max_pages * z.block + kTile - 1) / kTile;
    int64_t splits = num_sms / (ctas > 0 ? ctas : 1);
    if (splits > tiles / 2) splits = tiles / 2;
    r.splits = static_cast<int>(splits < 1 ? 1 : splits);
    return r;
}

cudaError_t launch_kv_attn_prefill(const KvAttn& a, const KvCache& c, const KvSteps& st, const KvPrefillPlan& plan,
                                   int row_min, void* workspace, cudaStream_t stream) {
    const PrefillArgs p = prefill_args(a, c, st, plan, row_min, workspace);
    if (c.D == 128)
        return c.mode == NV_KV_INT8 ? launch<NV_KV_INT8, 128>(p, stream) : launch<NV_KV_E4M3, 128>(p, stream);
    return c.mode == NV_KV_INT8 ? launch<NV_KV_INT8, 64>(p, stream) : launch<NV_KV_E4M3, 64>(p, stream);
}

cudaError_t launch_kv_attn_prefill_join(const KvAttn& a, const KvCache& c, const KvSteps& st, const KvPrefillPlan& plan,
                                        int row_min, void* workspace, cudaStream_t stream) {
    if (plan.splits <= 1) return cudaSuccess;
    const PrefillArgs p = prefill_args(a, c, st, plan, row_min, workspace);
    return c.D == 128 ? launch_join<128>(p, stream) : launch_join<64>(p, stream);
}

}  // namespace nvq
