// Attention of many query rows over the 4-bit paged cache (prompts, chunks) on
// the 5th-generation tensor cores.
//
// The rows of one sequence and key/value head (new tokens x heads of the group)
// are cut into items of 256: two tiles of 128 rows that share every key and value
// block. Per unit of 128 keys:
//   loader    (1 warp)   bulk copies of the block's packed codes and steps, page by
//                        page, into a ring;
//   unpack    (4 warps)  codes -> bf16 (one multiply-add a pair, exact, see kv4.cuh) in
//                        the 128-byte-swizzled layout: keys as K-major B operand, values
//                        as MN-major B operand, both row = token, so one routine does both.
//                        The 8 dims of a word are stored as the pairs (i, i + 4) that it
//                        unpacks into; the queries are stored in the same order, and the
//                        outputs are put back in order in registers.
//   MMA       (1 thread) S = Q K^T per tile into TMEM, O += P V with P from TMEM. The
//                        tiles take turns: while one tile's softmax runs, the tensor cores
//                        work on the other.
//   softmax   (2 x 4 warps) a thread owns a row: maximum, exponentials, denominator in
//                        fp32; P goes back to TMEM over S as bf16. O is rescaled only when a
//                        row's maximum grows by more than 2^8.
// Work split as in kv4_attn.cu: the units of all items in one line, an equal
// contiguous range per CTA (one CTA per SM), pieces of split items joined by a
// second kernel in a fixed order. Causal limits cut an item's blocks short.
//
// Every wait is bounded (1 s); one that gives up sets the device error word,
// lets the CTA drain and returns.
#include <algorithm>

#include "kv4.cuh"
#include "tc_ptx.cuh"

namespace bl {
namespace {

constexpr int BLK = 128;          // keys per unit
constexpr int TM = 128;           // rows per tile
constexpr int ROWS = 2 * TM;      // rows per item
constexpr int KV_STAGES = 4;      // unpacked tiles: K, V, K, V ...
constexpr int CODE_STAGES = 3;    // packed tiles
constexpr int THREADS = 512;
constexpr int MAX_CTAS = 148;     // sizes the workspace
constexpr int SEQ_GROUP = 32;     // sequences per entry of the coarse unit table
constexpr uint64_t WAIT_NS = 1000000000ull;
constexpr float RAISE = 8.0f;

struct TileArgs {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    Kv4View cache;
    Kv4Seqs batch;
    int M, group, max_q;
    float scale_log2;
    float* slots;   // [2 gridDim.x] pieces: [D / 4][ROWS] float4 sums, then [ROWS] (maximum, denominator)
    int4* joins;    // [gridDim.x]
    unsigned* err;
};

template <int D>
struct Cfg {
    static constexpr int TILE = BLK * D * 2;              // an unpacked K or V tile; also a Q tile
    static constexpr int CODES = BLK * D / 2;
    static constexpr int PACKED = CODES + BLK * (D / kKvGroup) * 2;
    static constexpr int HALF = BLK * 128;                // 64 dims of a tile
    static constexpr int SMEM = 1024 + (2 + KV_STAGES) * TILE + CODE_STAGES * PACKED;
    static constexpr int SLOT = ROWS * (D + 2);           // floats of a piece
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lbo_bytes >> 4) << 16;
    d |= static_cast<uint64_t>(sbo_bytes >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// bf16 inputs, fp32 accumulators; A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// A sequence's share of the work.
struct Seq {
    int row0, n_q, len, tiles;
};

__device__ __forceinline__ Seq seq_of(const TileArgs& a, int s, bool report) {
    Seq w;
    w.row0 = a.batch.q_start[s];
    const int end = a.batch.q_start[s + 1];
    w.n_q = end - w.row0;
    w.len = a.batch.kv_len[s];
    const int64_t room = (int64_t)a.batch.W << a.cache.page_shift;
    if (w.n_q <= 0 || w.row0 < 0 || end > a.M || w.n_q > a.max_q || w.len < 0 || w.len > room) {
        if (report && w.n_q != 0) atomicOr(a.err, kErrBadBatch);
        w.n_q = 0;
    }
    w.tiles = w.n_q > 0 ? (w.n_q * a.group + ROWS - 1) / ROWS : 0;
    return w;
}

// Blocks of item t of a sequence: up to the last key that its last row sees.
__device__ __forceinline__ int blocks_of(const TileArgs& a, const Seq& w, int t) {
    const int last = min(w.n_q - 1, ((t + 1) * ROWS - 1) / a.group);
    return max(1, (w.len - w.n_q + last + 1 + BLK - 1) / BLK);
}

__device__ __forceinline__ int units_of(const TileArgs& a, const Seq& w) {
    int n = 0;
    for (int t = 0; t < w.tiles; ++t) n += blocks_of(a, w, t);
    return n * a.cache.hkv;
}

// The pieces of this CTA's range, in order; every role walks its own copy.
struct Pieces {
    int u, u1;                      // next unit, end of the range
    int s, t, head, first, blocks;  // current item, its first unit
    Seq w;

    __device__ bool next(const TileArgs& a, int& b0, int& b1) {
        if (u >= u1) return false;
        while (u >= first + blocks) {  // move to the item that holds u
            first += blocks;
            if (++head == a.cache.hkv) {
                head = 0;
                if (++t >= w.tiles) {
                    t = 0;
                    do {
                        w = seq_of(a, ++s, false);
                    } while (w.tiles == 0);  // a later sequence has units: u < u1 <= total
                }
            }
            blocks = blocks_of(a, w, t);
        }
        b0 = u - first;
        b1 = min(blocks, b0 + (u1 - u));
        u += b1 - b0;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1) kv4_tile_kernel(const TileArgs a) {
    using C = Cfg<D>;
    constexpr int G = D / kKvGroup;
    constexpr int VB = D / 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * KV_STAGES + 2 * CODE_STAGES + 9];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    __shared__ int warp_sums[THREADS / 32];
    __shared__ int coarse[kKv4MaxSeqs / SEQ_GROUP + 1];  // units before each group of sequences
    __shared__ Pieces start_sh;
    __shared__ int total_sh;

    uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sT = sQ + 2 * C::TILE;
    uint8_t* sC = sT + KV_STAGES * C::TILE;
    auto bar = [&](int i) { return tc::smem_u32(bars + i); };
    auto tfull = [&](int i) { return bar(i); };
    auto tempty = [&](int i) { return bar(KV_STAGES + i); };
    auto cfull = [&](int i) { return bar(2 * KV_STAGES + i); };
    auto cempty = [&](int i) { return bar(2 * KV_STAGES + CODE_STAGES + i); };
    constexpr int B0 = 2 * KV_STAGES + 2 * CODE_STAGES;
    auto sfull = [&](int i) { return bar(B0 + i); };
    auto pfull = [&](int i) { return bar(B0 + 2 + i); };
    auto ofull = [&](int i) { return bar(B0 + 4 + i); };
    auto qfull = [&](int i) { return bar(B0 + 6 + i); };
    const uint32_t drained = bar(B0 + 8);  // teardown after an abort
    volatile int* aborted = &abort_sh;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < KV_STAGES; ++i) tc::mbar_init(tfull(i), 128), tc::mbar_init(tempty(i), 1);
        for (int i = 0; i < CODE_STAGES; ++i) tc::mbar_init(cfull(i), 1), tc::mbar_init(cempty(i), 128);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(sfull(i), 1);
            tc::mbar_init(pfull(i), 128);
            tc::mbar_init(ofull(i), 1);
            tc::mbar_init(qfull(i), 128);
        }
        tc::mbar_init(drained, 1);
        abort_sh = 0;
        tc::fence_mbar_init();
    }
    grid_dependency_wait();
    grid_dependents_launch();

    // ---- units of all sequences, and this CTA's range of them
    const int S = a.batch.S;
    {
        int carry = 0;
        for (int s0 = 0; s0 < S; s0 += THREADS) {
            const int s = s0 + tid;
            const int u = s < S ? units_of(a, seq_of(a, s, blockIdx.x == 0)) : 0;
            int sum = u;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) warp_sums[warp] = sum;
            __syncthreads();
            if (tid == 0)
                for (int w = 0; w < THREADS / 32 && s0 + w * SEQ_GROUP < S; ++w) {
                    coarse[s0 / SEQ_GROUP + w] = carry;
                    carry += warp_sums[w];
                }
            __syncthreads();
        }
        if (tid == 0) {
            coarse[(S + SEQ_GROUP - 1) / SEQ_GROUP] = carry;
            total_sh = carry;
            const int ctas = min((int)gridDim.x, carry);
            if ((int)blockIdx.x < ctas) {
                Pieces p;
                p.u = (int)((long long)carry * blockIdx.x / ctas);
                p.u1 = (int)((long long)carry * (blockIdx.x + 1) / ctas);
                int g = 0;
                while (coarse[g + 1] <= p.u) ++g;
                int before = coarse[g];
                for (p.s = g * SEQ_GROUP;; ++p.s) {
                    p.w = seq_of(a, p.s, false);
                    const int n = units_of(a, p.w);
                    if (before + n > p.u) break;
                    before += n;
                }
                for (p.t = 0;; ++p.t) {
                    p.blocks = blocks_of(a, p.w, p.t);
                    if (before + p.blocks * a.cache.hkv > p.u) break;
                    before += p.blocks * a.cache.hkv;
                }
                p.head = (p.u - before) / p.blocks;
                p.first = before + p.head * p.blocks;
                start_sh = p;
            }
        }
    }
    __syncthreads();
    const int total = total_sh;
    const int ctas = min((int)gridDim.x, total);
    const int c = blockIdx.x;
    if (c >= ctas) {
        if (tid == 0) a.joins[c] = make_int4(0, 0, 0, -1);
        return;
    }
    if (warp == 13) {
        tc::tmem_alloc(tc::smem_u32(&tmem_base_sh), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base_sh;
    const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 256 + D};
    auto give_up = [&]() {
        atomicOr(a.err, kErrTimeout);
        *aborted = 1;
    };

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 12) {
            // ------------------------------------------------------------ loader
            // the cache may have been written by ordinary stores of the kernel before
            asm volatile("fence.proxy.async.global;" ::: "memory");
            Pieces p = start_sh;
            const int shift = a.cache.page_shift;
            const int part_keys = min(BLK, 1 << shift);
            const int parts = BLK / part_keys;
            uint32_t g = 0;  // packed tiles so far
            int b0, b1;
            bool ok = true;
            while (ok && p.next(a, b0, b1)) {
                const int* row = a.batch.table + p.s * a.batch.table_stride;
                int have = -1, page = 0;
                for (int b = b0; b < b1 && ok; ++b) {
                    const int p0 = b * parts;
                    if (have < 0 || p0 - have + parts > 32) {
                        have = p0;
                        const int key = (p0 + lane) * part_keys;
                        page = 0;
                        if (key < p.w.len) {
                            page = row[key >> shift];
                            if (page < 0 || page >= a.cache.num_pages) {
                                atomicOr(a.err, kErrBadBatch);
                                page = 0;  // an existing page stands in: the rows are unspecified
                            }
                        }
                    }
                    const int live = max(0, min(parts, (p.w.len - b * BLK + part_keys - 1) / part_keys));
#pragma unroll 1
                    for (int v = 0; v < 2; ++v, ++g) {
                        const int st = g % CODE_STAGES;
                        if (g >= CODE_STAGES) ok = tc::mbar_wait(cempty(st), (g / CODE_STAGES - 1) & 1, WAIT_NS);
                        ok = __all_sync(0xffffffffu, ok && !*aborted);
                        if (!ok) break;
                        if (lane == 0) tc::mbar_arrive_expect_tx(cfull(st), live * part_keys * (VB + 2 * G));
                        __syncwarp();
                        const int part = lane >> 1, steps = lane & 1;
                        const int pg = __shfl_sync(0xffffffffu, page, (p0 - have + part) & 31);
                        if (part < live) {
                            const int64_t vec = (((int64_t)pg * a.cache.hkv + p.head) << shift) + ((b * BLK + part * part_keys) & ((1 << shift) - 1));
                            const uint32_t base = tc::smem_u32(sC + st * C::PACKED);
                            if (steps)
                                bulk_copy(base + C::CODES + part * part_keys * 2 * G, (v ? a.cache.vs : a.cache.ks) + vec * G, part_keys * 2 * G, cfull(st));
                            else
                                bulk_copy(base + part * part_keys * VB, (v ? a.cache.vc : a.cache.kc) + vec * VB, part_keys * VB, cfull(st));
                        }
                    }
                }
            }
            if (!ok && lane == 0) {
                give_up();
                // let the copies still in flight land before the CTA exits
                for (uint32_t h = g > CODE_STAGES ? g - CODE_STAGES : 0; h < g; ++h)
                    tc::mbar_wait(cfull(h % CODE_STAGES), (h / CODE_STAGES) & 1, WAIT_NS);
            }
        } else if (warp == 13 && lane == 0) {
            // ------------------------------------------------------------ MMA issuer
            constexpr uint32_t id_s = idesc_bf16(TM, BLK, false);
            constexpr uint32_t id_o = idesc_bf16(TM, D, true);
            Pieces p = start_sh;
            uint32_t n = 0;                    // blocks so far (K tile 2n, V tile 2n + 1 of the ring)
            uint32_t np[2] = {0, 0};           // P tiles consumed
            uint32_t nq[2] = {0, 0};           // Q tiles consumed
            int b0, b1;
            bool ok = true;
            auto wait = [&](uint32_t b, uint32_t parity) { return ok && !*aborted && tc::mbar_wait(b, parity, WAIT_NS); };
            auto scores = [&](int i, uint32_t kt) {
                const uint64_t qd = desc_sw128(tc::smem_u32(sQ + i * C::TILE), 16, 1024);
                const uint64_t kd = desc_sw128(tc::smem_u32(sT + (kt % KV_STAGES) * C::TILE), 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k / 4) * C::HALF + (k % 4) * 32) >> 4;
                    mma_ss(tS[i], qd + off, kd + off, id_s, k != 0);
                }
                tc::mma_commit(sfull(i));
            };
            auto values = [&](int i, uint32_t vt, bool first) {
                const uint64_t vd = desc_sw128(tc::smem_u32(sT + (vt % KV_STAGES) * C::TILE), C::HALF, 1024);
#pragma unroll
                for (int k = 0; k < BLK / 16; ++k)
                    mma_ts(tO[i], tS[i] + 8 * k, vd + ((k * 16 * 128) >> 4), id_o, !first || k != 0);
            };
            while (ok && p.next(a, b0, b1)) {
                const bool two = p.w.n_q * a.group - p.t * ROWS > TM;
                const int cnt = b1 - b0;
                for (int j = -1; j < cnt && ok; ++j, ++n) {
                    const bool more = j + 1 < cnt;
                    const uint32_t vt = 2 * (n - 1) + 1, kt = 2 * n;  // V of block j, K of block j + 1
                    if (j >= 0) ok = wait(tfull(vt % KV_STAGES), (vt / KV_STAGES) & 1);
                    if (more) ok = wait(tfull(kt % KV_STAGES), (kt / KV_STAGES) & 1);
                    if (!ok) break;
#pragma unroll 1
                    for (int i = 0; i < (two ? 2 : 1) && ok; ++i) {
                        if (j >= 0) {
                            ok = wait(pfull(i), np[i] & 1);
                            if (!ok) break;
                            ++np[i];
                            tc::fence_after_sync();
                            values(i, vt, j == 0);
                            if (!more) tc::mma_commit(ofull(i));
                        } else {
                            ok = wait(qfull(i), nq[i] & 1);
                            if (!ok) break;
                            ++nq[i];
                            tc::fence_after_sync();
                        }
                        if (i == (two ? 1 : 0) && j >= 0) tc::mma_commit(tempty(vt % KV_STAGES));
                        if (more) scores(i, kt);
                    }
                    if (ok && more) tc::mma_commit(tempty(kt % KV_STAGES));
                    if (!more) break;  // n already counts this piece's blocks
                }
            }
            if (!ok) give_up();
        }
    } else if (warp >= 8) {
        // ---------------------------------------------------------------- unpack
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        Pieces p = start_sh;
        const int t = lane & 3;
        const int row = (warp - 8) * 8 + (lane >> 2);  // key of the pass
        uint32_t g = 0;
        int b0, b1;
        bool ok = true;
        while (ok && p.next(a, b0, b1)) {
            for (int b = b0; b < b1 && ok; ++b) {
#pragma unroll 1
                for (int v = 0; v < 2; ++v, ++g) {
                    const int cs = g % CODE_STAGES, ts = g % KV_STAGES;
                    ok = !*aborted && tc::mbar_wait(cfull(cs), (g / CODE_STAGES) & 1, WAIT_NS) &&
                         (g < KV_STAGES || tc::mbar_wait(tempty(ts), (g / KV_STAGES - 1) & 1, WAIT_NS));
                    if (!ok) {
                        give_up();
                        break;
                    }
                    const uint8_t* codes = sC + cs * C::PACKED;
                    uint8_t* tile = sT + ts * C::TILE;
#pragma unroll
                    for (int pass = 0; pass < 4; ++pass) {
                        const int key = pass * 32 + row;
                        uint32_t w[G], st[G];
                        if constexpr (D == 128) {
                            const uint4 x = *reinterpret_cast<const uint4*>(codes + key * VB + 16 * t);
                            const uint2 y = *reinterpret_cast<const uint2*>(codes + C::CODES + key * 2 * G);
                            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
                            st[0] = __byte_perm(y.x, 0, 0x1010), st[1] = __byte_perm(y.x, 0, 0x3232);
                            st[2] = __byte_perm(y.y, 0, 0x1010), st[3] = __byte_perm(y.y, 0, 0x3232);
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(codes + key * VB + 8 * t);
                            const uint32_t y = *reinterpret_cast<const uint32_t*>(codes + C::CODES + key * 2 * G);
                            w[0] = x.x, w[1] = x.y;
                            st[0] = __byte_perm(y, 0, 0x1010), st[1] = __byte_perm(y, 0, 0x3232);
                        }
                        if (b * BLK + key >= p.w.len) {  // behind the last token: whatever the page holds
#pragma unroll
                            for (int e = 0; e < G; ++e) st[e] = 0;
                        }
                        // odd keys take their groups in swapped order, so that the 8 lanes of a store phase
                        // cover all 8 chunks of a 128-byte row
                        const bool odd = key & 1;
                        uint8_t* base = tile + key * 128;
#pragma unroll
                        for (int e = 0; e < G; ++e) {
                            const uint32_t word = odd ? w[e ^ 1] : w[e], s = odd ? st[e ^ 1] : st[e];
                            const int gr = e ^ (odd ? 1 : 0);
                            const uint32_t s16 = bf16x2_mul(s, kBf16x2Sixteen), s24 = bf16x2_mul(s, kBf16x2MinusTwentyFour);
                            const uint4 o = make_uint4(bf16x2_fma(kv4_unit_pair<0>(word), s16, s24), bf16x2_fma(kv4_unit_pair<1>(word), s16, s24),
                                                       bf16x2_fma(kv4_unit_pair<2>(word), s16, s24), bf16x2_fma(kv4_unit_pair<3>(word), s16, s24));
                            const int chunk = 4 * (gr & 1) + t;
                            *reinterpret_cast<uint4*>(base + (e >> 1) * C::HALF + ((chunk ^ (key & 7)) << 4)) = o;
                        }
                    }
                    tc::mbar_arrive(cempty(cs));
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(tfull(ts));
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax: tile i, row r of it
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int i = warp >> 2, r = tid & (TM - 1);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float sc = a.scale_log2;
        Pieces p = start_sh;
        uint32_t ns = 0, no = 0;
        int4 join = make_int4(0, 0, 0, -1);
        int b0, b1;
        bool ok = true;
        while (ok && p.next(a, b0, b1)) {
            const int rows = min(ROWS, p.w.n_q * a.group - p.t * ROWS);
            const bool starts = b0 == 0, ends = b1 == p.blocks;
            if (starts && !ends) {
                const int item_end = p.first + p.blocks;
                const int last = (int)(((long long)item_end * ctas + total - 1) / total) - 1;
                join = make_int4(p.w.row0, p.head, p.t | (rows << 20), last);
            }
            if (i * TM >= rows) continue;
            const int ri = p.t * ROWS + i * TM + r;  // row of the sequence
            const bool live = i * TM + r < rows;
            const int token = ri / a.group, qh = p.head * a.group + ri % a.group;
            const int limit = live ? min(p.w.len, p.w.len - p.w.n_q + token + 1) : 0;
            const int least = p.w.len - p.w.n_q + (p.t * ROWS + i * TM) / a.group + 1;  // keys all rows see
            {   // this row's queries -> shared memory
                const uint16_t* qp = a.q + (live ? (int64_t)(p.w.row0 + token) * a.q_stride + qh * D : 0);
                uint8_t* dst = sQ + i * C::TILE + r * 128;
#pragma unroll
                for (int o = 0; o < D / 8; ++o) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (live) x = *reinterpret_cast<const uint4*>(qp + 8 * o);
                    const uint4 y = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                                               __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
                    *reinterpret_cast<uint4*>(dst + (o >> 3) * C::HALF + (((o & 7) ^ (r & 7)) << 4)) = y;
                }
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(qfull(i));
            }
            float mx = -INFINITY, thr = -INFINITY, msc = 0.0f, den = 0.0f;
            for (int b = b0; b < b1; ++b, ++ns) {
                ok = !*aborted && tc::mbar_wait(sfull(i), ns & 1, WAIT_NS);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after_sync();
                uint32_t s[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tc::tmem_ld_32x32(tS[i] + lanes + 32 * k, s[k]);
                tc::tmem_ld_wait();
                if (b * BLK + BLK > least) {
                    const int seen = limit - b * BLK;  // columns this row sees
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (32 * k + x >= seen) s[k][x] = 0xFF800000u;
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < 32; ++x)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], __uint_as_float(s[k][x]));
                const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                const bool raise = m > thr;
                if (__any_sync(0xffffffffu, raise)) {
                    float f = 1.0f;
                    if (raise) {
                        const float now = m * sc;
                        f = mx == -INFINITY ? 0.0f : exp2_approx(msc - now);
                        mx = m;
                        msc = now;
                        thr = m + RAISE / sc;
                        den *= f;
                    }
                    if (b > b0) {  // the block before has been added: its MMA finished before this S
#pragma unroll 1
                        for (int k = 0; k < D / 32; ++k) {
                            uint32_t o[32];
                            tc::tmem_ld_32x32(tO[i] + lanes + 32 * k, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tc::tmem_st_32x32(tO[i] + lanes + 32 * k, o);
                        }
                    }
                }
                float d4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        const int k = 2 * h + (x >> 4), y = 2 * (x & 15);
                        const float p0 = exp2_approx(fmaf(__uint_as_float(s[k][y]), sc, -msc));
                        const float p1 = exp2_approx(fmaf(__uint_as_float(s[k][y + 1]), sc, -msc));
                        d4[2 * (x & 1)] += p0;
                        d4[2 * (x & 1) + 1] += p1;
                        pk[x] = pack_bf16(p0, p1);
                    }
                    tc::tmem_st_32x32(tS[i] + lanes + 32 * h, pk);
                }
                den += (d4[0] + d4[1]) + (d4[2] + d4[3]);
                tc::tmem_st_wait();
                tc::fence_before_sync();
                tc::mbar_arrive(pfull(i));
            }
            if (ok) {
                ok = !*aborted && tc::mbar_wait(ofull(i), no & 1, WAIT_NS);
                ok = __all_sync(0xffffffffu, ok);
                ++no;
            }
            if (!ok) {
                give_up();
                break;
            }
            tc::fence_after_sync();
            const bool whole = starts && ends;
            const float inv = den == 0.0f ? 0.0f : 1.0f / den;
            float4* slot = reinterpret_cast<float4*>(a.slots + (size_t)(2 * c + (starts ? 1 : 0)) * C::SLOT) + i * TM + r;
            uint16_t* op = a.out + (live ? (int64_t)(p.w.row0 + token) * a.out_stride + qh * D : 0);
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
                uint32_t o[32];
                tc::tmem_ld_32x32(tO[i] + lanes + 32 * k, o);
                tc::tmem_ld_wait();
                if (!live) continue;
#pragma unroll
                for (int x = 0; x < 32; x += 8) {
                    float f[8];  // back in order: column 2j is dim j, column 2j + 1 dim j + 4
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f[j] = __uint_as_float(o[x + 2 * j]);
                        f[j + 4] = __uint_as_float(o[x + 2 * j + 1]);
                    }
                    if (whole) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] *= inv;
                        *reinterpret_cast<uint4*>(op + 32 * k + x) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
                    } else {
                        slot[(8 * k + x / 4) * ROWS] = make_float4(f[0], f[1], f[2], f[3]);
                        slot[(8 * k + x / 4 + 1) * ROWS] = make_float4(f[4], f[5], f[6], f[7]);
                    }
                }
            }
            if (!whole && live) {
                float2* st = reinterpret_cast<float2*>(a.slots + (size_t)(2 * c + (starts ? 1 : 0)) * C::SLOT + ROWS * D) + i * TM + r;
                *st = make_float2(mx == -INFINITY ? -INFINITY : msc, den);
            }
        }
        if (tid == 0) a.joins[c] = ok ? join : make_int4(0, 0, 0, -1);
    }

    // -------------------------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 13) {
        if (lane == 0 && abort_sh) {
            // no MMA may still be using TMEM when it is released
            tc::mma_commit(drained);
            tc::mbar_wait(drained, 0, WAIT_NS);
        }
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Join the pieces of split items: block (c, y) takes part y of the [D / 4][ROWS]
// sums of the item whose first piece CTA c held.
template <int D>
__global__ void __launch_bounds__(ROWS) kv4_tile_join_kernel(const TileArgs a) {
    using C = Cfg<D>;
    grid_dependency_wait();
    grid_dependents_launch();
    const int4 j = a.joins[blockIdx.x];
    const int c = blockIdx.x, row = threadIdx.x;
    const int rows = j.z >> 20, t = j.z & 0xfffff;
    if (j.w < 0 || row >= rows) return;
    const int pieces = j.w - c + 1;
    auto slot = [&](int p) { return a.slots + (size_t)(2 * (c + p) + (p == 0 ? 1 : 0)) * C::SLOT; };
    float m = -INFINITY;
    for (int p = 0; p < pieces; ++p) m = fmaxf(m, slot(p)[ROWS * D + 2 * row]);
    float den = 0.0f;
    float4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int p = 0; p < pieces; ++p) {
        const float* sp = slot(p);
        const float2 st = reinterpret_cast<const float2*>(sp + ROWS * D)[row];
        const float f = st.x == -INFINITY ? (st.y != st.y ? 1.0f : 0.0f) : exp2_approx(st.x - m);
        den += f * st.y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 o = reinterpret_cast<const float4*>(sp)[(4 * blockIdx.y + e) * ROWS + row];
            v[e].x += f * o.x, v[e].y += f * o.y, v[e].z += f * o.z, v[e].w += f * o.w;
        }
    }
    const float inv = den == 0.0f ? 0.0f : 1.0f / den;
    const int ri = t * ROWS + row;
    uint16_t* op = a.out + (int64_t)(j.x + ri / a.group) * a.out_stride + (j.y * a.group + ri % a.group) * D + 16 * blockIdx.y;
#pragma unroll
    for (int e = 0; e < 4; e += 2)
        *reinterpret_cast<uint4*>(op + 4 * e) =
            make_uint4(pack_bf16(v[e].x * inv, v[e].y * inv), pack_bf16(v[e].z * inv, v[e].w * inv),
                       pack_bf16(v[e + 1].x * inv, v[e + 1].y * inv), pack_bf16(v[e + 1].z * inv, v[e + 1].w * inv));
}

template <int D>
cudaError_t launch_tile(const TileArgs& args, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static int sms[64];
    if (dev >= 64 || !sms[dev]) {
        e = cudaFuncSetAttribute(kv4_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
        int n = 0;
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (dev < 64) sms[dev] = n;
    }
    const int grid = std::min(MAX_CTAS, dev < 64 ? sms[dev] : MAX_CTAS);
    e = launch_pdl(kv4_tile_kernel<D>, dim3((unsigned)grid), dim3(THREADS), Cfg<D>::SMEM, s, args);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv4_tile_join_kernel<D>, dim3((unsigned)grid, D / 16), dim3(ROWS), 0, s, args);
}

}  // namespace

size_t kv4_tile_workspace_bytes(int D) {
    return (size_t)2 * MAX_CTAS * ROWS * (D + 2) * 4 + (size_t)MAX_CTAS * sizeof(int4);
}

cudaError_t launch_kv4_tile(const uint16_t* q, int64_t q_stride, int64_t M, int Hq, int D, int64_t max_q, float scale,
                            const Kv4View& cache, const Kv4Seqs& batch, uint16_t* out, int64_t out_stride, void* ws,
                            cudaStream_t s) {
    TileArgs a;
    a.q = q, a.out = out, a.q_stride = q_stride, a.out_stride = out_stride;
    a.cache = cache, a.batch = batch;
    a.M = (int)M, a.group = Hq / cache.hkv, a.max_q = (int)std::min<int64_t>(max_q, M);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.slots = (float*)ws;
    a.joins = (int4*)((char*)ws + (size_t)2 * MAX_CTAS * ROWS * (D + 2) * 4);
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    return D == 128 ? launch_tile<128>(a, s) : launch_tile<64>(a, s);
}

}  // namespace bl
