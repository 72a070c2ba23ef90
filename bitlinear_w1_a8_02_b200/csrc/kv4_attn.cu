// Attention of few query rows over the 4-bit paged cache (decode).
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale (q . k_j) - max)
//
// Bound by the cache's bytes (144 a key and head at D = 128), so every key is
// read once for all query heads that share it and the unpacking has to keep up.
// The query rows of one sequence and key/value head (new tokens x heads of the
// group, at most 8 NT) are the n of mma.sync m16n8k16:
//   scores   S^T [16 keys x rows] = K [16 x D] Q^T: a thread's 16 bytes of a key
//            hold an octet of each group, so each pair of k-steps stays inside one
//            group. The nibbles enter as bf16 subnormals (an AND and half a shift a
//            pair, see raw_pair); the accumulator starts at -8 sum q, which leaves
//            sum c q, and the step multiplies once per key and group.
//   values   O^T [D x rows] += V^T [D x 16 keys] P^T: pairs of keys are brought
//            together by byte permutes of the packed words, then one AND/OR and one
//            multiply-add give the bf16 pair exactly (see kv4.cuh); P^T comes from the
//            score registers by an 8x8 transpose.
// A running maximum is kept per row and only raised when a score passes it by
// 2^8 (in the exponent's base-2 units), so accumulators are rarely rescaled. It is
// taken off the scores before they are scaled: one multiply-add with the scaled
// maximum would leave that one's rounding, which passes the exponent's range for
// scores of 2^31 and more. (Two instructions a score instead of one, 0.9% of the
// time; a branch for the rows that need it cost 1.5%.)
//
// Work split: all (sequence, head, row block) items are cut into units of 128
// keys and every CTA takes one contiguous range of units, whatever the lengths
// are. A CTA that holds a whole item writes its rows; a piece goes to the CTA's
// slot in the workspace as unnormalised sums, maximum and denominator, and a
// second kernel joins the pieces in order. Four warps take 32 keys of a unit
// each; a fifth copies the units' pages into a ring (bulk copies, the page ids
// of 32 copies ahead loaded at once).
//
// The weights p_j are rounded to bf16 for the product with the values (2^-8 each, which
// averages out over the keys): the tensor cores take no wider operand beside bf16 values.
// The denominator sums them as they are.
//
// Measured (20 query, 5 key/value heads of 128): 64 sequences of 8192 keys 101 us with
// cold caches, 3.7 TB/s of cache, 57% of the issue slots, 55% of the ALU's. A copy without
// the loads takes as long, so memory is not the bound; neither pipe is full, so what bounds
// it is the chain of a warp's 16 keys (scores, vote, exponentials, transpose, values) with
// only 12 warps on an SM to hide it, 8 with more than 8 rows. 64 sequences of 2048
// keys: 36 us with 5 rows a head, 55 with 16. One sequence of 4001 keys: 10.1 us, units
// and joins about half each. Other splits measured slower: 8 warps a block, 3 stages,
// 4 blocks an SM.
#include <algorithm>

#include <cfloat>
#include <cmath>

#include "kv4.cuh"
#include "tc_ptx.cuh"

namespace bl {
namespace {

constexpr int kKeys = 128;       // keys per unit
constexpr int kWarps = 4;        // consumer warps, 32 keys of a unit each, 16 at a time
constexpr int kWarpKeys = kKeys / kWarps;
constexpr int kThreads = 32 * (kWarps + 1);
// What starting and ending an item costs, in units (it evens out the ranges): 64 x 2048 keys 35.0 us with 2, 36.3 with
// 1, 37.7 with 4; 8 x 600 keys 13.8 with 2, 15.2 with 4.
constexpr int kItemUnits = 2;
constexpr int kStages = 2;
constexpr int kMaxCtas = 592;    // four per SM on 148 SMs; sizes the workspace
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kGaveUp = -2;
constexpr float kRaise = 8.0f;   // a maximum is raised when a score passes it by this (base 2)

struct RowsArgs {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    Kv4View cache;
    Kv4Seqs batch;
    int M, group, max_q;  // query heads per key/value head
    float scale_log2;     // scale * log2(e)
    int least_shift;      // of the queries' scaling, so that scale_log2 * 2^(kSpacing - shift) stays below 2^127
    float* slots;         // [2 gridDim.x][8 NT][D + 2]: sums, maximum, denominator of pieces
    int4* joins;          // [gridDim.x]: item whose first piece the CTA holds: first row, head, row block | rows << 24, last CTA;
                          // .w = -1: none, kGaveUp: none, and its own pieces are not all there
    unsigned* err;
};

template <int D>
struct Stage {
    static constexpr int CODES = kKeys * D / 2;
    static constexpr int STEPS = kKeys * (D / kKvGroup) * 2;
    static constexpr int BYTES = 2 * (CODES + STEPS);  // kc, vc, ks, vs
};

template <int D, int NT>
struct RowsSmem {
    static constexpr int MERGE = kWarps * 8 * NT * D * 4;  // a warp's unnormalised sums
    static constexpr int STATS = kWarps * 8 * NT * 2 * 4;
    static constexpr int FIXED = kStages * Stage<D>::BYTES + MERGE + STATS + 2 * kStages * 8 + 64;
    static size_t bytes(int S) { return FIXED + (size_t)(S + 1) * 4; }
};

// tc::mbar_wait with a hint that lets the warp sleep up to 20 us at a time: the polls of waiting warps take issue
// slots from the unpacking ones.
__device__ __forceinline__ bool mbar_wait_asleep(uint32_t bar, uint32_t parity) {
    return bounded_wait<1>(
        [&] {
            uint32_t ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\tselp.b32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(bar), "r"(parity)
                : "memory");
            return ok != 0;
        },
        [] { return tc::globaltimer_ns(); }, kWaitLimitNs);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with an accumulator operand of its own: rows r and r + 8 both start from (c0, c1).
__device__ __forceinline__ void mma_bf16_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Nibbles I, I + 4 of a word as a bf16 pair without any arithmetic: a bf16's low 8 bits are linear (the subnormals and
// the first normal binade have one spacing), so bits 0..3 are n 2^-133 and bits 4..7 16 n 2^-133; the tensor cores take
// subnormals. Odd I come out 16 times as large, which the queries make up for.
template <int I>
__device__ __forceinline__ uint32_t raw_pair(uint32_t w) {
    const uint32_t x = I < 2 ? w : w >> 8;
    return x & (I & 1 ? 0x00F000F0u : 0x000F000Fu);
}

constexpr int kSpacing = 133;  // -log2 of the spacing of bf16's subnormals

// A maximum in the exponent's units. Below fp32 it weighs nothing, but is no NaN; above, the infinity makes its row NaN
// where pieces meet.
__device__ __forceinline__ float in_units(float m, float sc) { return fmaxf(m * sc, -FLT_MAX); }

// Barrier of the consumer warps that tells all of them whether any thread of theirs came with `p`.
__device__ __forceinline__ bool consumers_meet(bool p) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)p), "n"(32 * kWarps)
        : "memory");
    return any != 0;
}

// Units of kKeys keys of sequence s (0 when it has no new tokens or was refused).
struct SeqWork {
    int n_q, len, row0, blocks, row_blocks;
};

template <int RB>
__device__ __forceinline__ SeqWork seq_work(const RowsArgs& a, int s, bool report) {
    SeqWork w;
    w.row0 = a.batch.q_start[s];
    const int end = a.batch.q_start[s + 1];
    w.n_q = end - w.row0;
    w.len = a.batch.kv_len[s];
    const int64_t room = (int64_t)a.batch.W << a.cache.page_shift;
    if (w.n_q <= 0 || w.row0 < 0 || end > a.M || w.n_q > a.max_q || w.len < 0 || w.len > room) {
        if (report && w.n_q != 0) atomicOr(a.err, kErrBadBatch);
        w.n_q = 0;
    }
    w.blocks = max(1, (w.len + kKeys - 1) / kKeys);  // an empty cache: one unit without keys writes the zeros
    w.row_blocks = w.n_q ? (w.n_q * a.group + RB - 1) / RB : 0;
    return w;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) kv4_rows_kernel(const RowsArgs a) {
    constexpr int G = D / kKvGroup;
    constexpr int RB = 8 * NT;
    constexpr int VB = D / 2;  // bytes of a packed vector
    constexpr int MT = D / 16;  // 16-dim tiles of the output
    using St = Stage<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* merge = reinterpret_cast<float*>(ring + kStages * St::BYTES);
    float* stats = merge + kWarps * RB * D;
    uint64_t* bars = reinterpret_cast<uint64_t*>(stats + kWarps * RB * 2);
    int* scratch = reinterpret_cast<int*>(bars + 2 * kStages);  // 16 ints
    int* prefix = scratch + 16;                                 // [S + 1] units before sequence s
    auto full = [&](int i) { return tc::smem_u32(bars + i); };
    auto empty = [&](int i) { return tc::smem_u32(bars + kStages + i); };
    volatile int* abort_flag = scratch + 15;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(full(i), 1);
            tc::mbar_init(empty(i), kWarps);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    grid_dependency_wait();
    grid_dependents_launch();
    // the cache may have been written by ordinary stores of the kernel before
    asm volatile("fence.proxy.async.global;" ::: "memory");

    // units before each sequence
    const int S = a.batch.S, hkv = a.cache.hkv;
    int carry = 0;
    for (int s0 = 0; s0 < S; s0 += kThreads) {
        const int s = s0 + tid;
        int u = 0;
        if (s < S) {
            const SeqWork w = seq_work<RB>(a, s, blockIdx.x == 0);
            u = hkv * w.row_blocks * (kItemUnits + w.blocks);
        }
        int sum = u;  // inclusive over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += t;
        }
        if (lane == 31) scratch[warp] = sum;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < kWarps + 1; ++w) {
            if (w < warp) before += scratch[w];
            carry += scratch[w];
        }
        if (s < S) prefix[s] = before + sum - u;
        __syncthreads();
    }
    if (tid == 0) prefix[S] = carry;
    __syncthreads();
    const int total = carry;
    const int ctas = min((int)gridDim.x, total);
    if ((int)blockIdx.x >= ctas) {
        if (tid == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, -1);
        return;
    }
    const int c = blockIdx.x;
    const int u0 = (int)((long long)total * c / ctas), u1 = (int)((long long)total * (c + 1) / ctas);

    // The item that holds unit u: sequence by binary search, then head and row block.
    struct Item {
        int s, head, rb, first, end;  // units of its blocks; those that stand for its cost come before
        SeqWork w;
    };
    auto find = [&](int u) {
        int lo = 0, hi = S - 1;  // the last s with prefix[s] <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        Item it;
        it.s = lo;
        it.w = seq_work<RB>(a, lo, false);
        const int span = kItemUnits + it.w.blocks;
        const int j = (u - prefix[lo]) / span;
        it.rb = j % it.w.row_blocks;
        it.head = j / it.w.row_blocks;
        it.first = prefix[lo] + j * span + kItemUnits;
        it.end = it.first + it.w.blocks;
        return it;
    };

    if (warp == kWarps) {
        // ------------------------------------------------------------ producer
        const int shift = a.cache.page_shift;
        const int part_keys = min(kKeys, 1 << shift);
        const int parts = kKeys / part_keys;  // copies of one array per unit
        int g = 0;
        bool ok = true;
        for (int u = u0; u < u1 && ok;) {
            const Item it = find(u);
            const int end = min(u1, it.end);
            u = max(u, it.first);  // not past u1 by more than the item's cost: then there is no block here
            const int* row = a.batch.table + it.s * a.batch.table_stride;
            // page of part p (32 parts ahead, one per lane)
            int have = -1, page = 0;
            for (; u < end; ++u, ++g) {
                const int blk = u - it.first, st = g % kStages;
                const int p0 = blk * parts;
                if (have < 0 || p0 - have + parts > 32) {
                    have = p0;
                    const int key = (p0 + lane) * part_keys;
                    page = 0;
                    if (key < it.w.len) {
                        page = row[key >> shift];
                        if (page < 0 || page >= a.cache.num_pages) {
                            atomicOr(a.err, kErrBadBatch);
                            page = 0;  // an existing page stands in: the rows are unspecified
                        }
                    }
                }
                if (g >= kStages) ok = mbar_wait_asleep(empty(st), (g / kStages - 1) & 1);
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                if (!ok) break;
                const int live = min(parts, (it.w.len - blk * kKeys + part_keys - 1) / part_keys);
                const uint32_t bytes = live * part_keys * (VB + 2 * G) * 2;
                if (lane == 0) tc::mbar_arrive_expect_tx(full(st), bytes);
                __syncwarp();
                const int part = lane >> 2, array = lane & 3;
                const int pg = __shfl_sync(0xffffffffu, page, (p0 - have + part) & 31);
                if (part < live) {
                    const int64_t vec = (((int64_t)pg * hkv + it.head) << shift) + ((blk * kKeys + part * part_keys) & ((1 << shift) - 1));
                    const uint32_t base = tc::smem_u32(ring + st * St::BYTES);
                    if (array < 2)
                        bulk_copy(base + array * St::CODES + part * part_keys * VB,
                                  (array ? a.cache.vc : a.cache.kc) + vec * VB, part_keys * VB, full(st));
                    else
                        bulk_copy(base + 2 * St::CODES + (array - 2) * St::STEPS + part * part_keys * G * 2,
                                  (array == 3 ? a.cache.vs : a.cache.ks) + vec * G, part_keys * G * 2, full(st));
                }
            }
        }
        if (lane == 0) {
            if (!ok) {
                atomicOr(a.err, kErrTimeout);
                *abort_flag = 1;
            }
            // let the copies still in flight land before the CTA exits: the consumers wait for them too, unless they give up
            for (int h = max(0, g - kStages); h < g; ++h) mbar_wait_asleep(full(h % kStages), (h / kStages) & 1);
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int r = lane >> 2, t = lane & 3;
    const int kr = r ^ ((r >> 1) & 1);  // key of score row r: neighbours in one order or the other, so that the keys a value
                                        // load takes for t = 0 .. 3 are even and odd ones (two bank halves)
    int g = 0;
    int4 join = make_int4(0, 0, 0, -1);
    for (int u = u0; u < u1;) {
        const Item it = find(u);
        const int end = min(u1, it.end);
        u = max(u, it.first);
        if (u >= end) continue;  // the range ends inside the item's cost
        const int rows = min(RB, it.w.n_q * a.group - it.rb * RB);
        const int begin = u;

        // Queries of this lane's rows (columns r of each n-tile) in the order of the nibbles, scaled by a power of two
        // per row that brings the largest to 2^100 .. 2^101 (exact: products with n 2^-133 stay far from fp32's ends),
        // and -8 sum q, which the accumulators of a group start from: they end as sum c q.
        uint32_t qf[NT][G][4];
        float c0[NT][G][4];
        float sc[NT][2];  // of accumulator columns 2t, 2t + 1: softmax scale * log2(e), the rows' scaling taken back
        int lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = nt * 8 + r;
            const int ri = it.rb * RB + row;
            const bool live = row < rows;
            const uint16_t* qp = a.q + (live ? (int64_t)(it.w.row0 + ri / a.group) * a.q_stride + (it.head * a.group + ri % a.group) * D : 0);
            uint32_t top = 0;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (live) x = *reinterpret_cast<const uint4*>(qp + 32 * gr + 8 * t);
                qf[nt][gr][0] = __byte_perm(x.x, x.z, 0x5410);
                qf[nt][gr][1] = __byte_perm(x.x, x.z, 0x7632);
                qf[nt][gr][2] = __byte_perm(x.y, x.w, 0x5410);
                qf[nt][gr][3] = __byte_perm(x.y, x.w, 0x7632);
#pragma unroll
                for (int i = 0; i < 4; ++i) top = __vmaxu2(top, qf[nt][gr][i] & 0x7FFF7FFFu);
            }
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int shift = min(127, max(a.least_shift, 227 - (int)(top >> 7)));
            const uint32_t even = (uint32_t)(127 + shift) << 7, odd = (uint32_t)(123 + shift) << 7;
            const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum += __uint_as_float(qf[nt][gr][i] << 16) + __uint_as_float(qf[nt][gr][i] & 0xffff0000u);
                    const uint32_t f = i & 1 ? odd : even;
                    qf[nt][gr][i] = bf16x2_mul(qf[nt][gr][i], f | f << 16);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum = sum * up * -0x1p-65f * 0x1p-65f;  // -8 * 2^-133
                c0[nt][gr][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
                c0[nt][gr][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
                c0[nt][gr][2] = c0[nt][gr][0], c0[nt][gr][3] = c0[nt][gr][1];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                sc[nt][e] = a.scale_log2 * __uint_as_float((uint32_t)(127 + kSpacing - __shfl_sync(0xffffffffu, shift, 8 * t + 4 * e)) << 23);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rc = it.rb * RB + nt * 8 + 2 * t + e;  // row of accumulator column e
                lim[nt][e] = min(it.w.len, it.w.len - it.w.n_q + rc / a.group + 1);
            }
        }
        const int least = it.w.len - it.w.n_q + (it.rb * RB) / a.group + 1;  // keys every row sees

        float o[NT][MT][4];
        float mx[NT][2], thr[NT][2], ref[NT][2], den[NT][2];  // ref: the maximum, 0 while there is none
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[nt][e] = thr[nt][e] = -INFINITY, ref[nt][e] = den[nt][e] = 0.0f;
        }

        bool ok = true;
        for (; u < end; ++u, ++g) {
            const int st = g % kStages;
            ok = mbar_wait_asleep(full(st), (g / kStages) & 1) && !*abort_flag;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int sub = 0; sub < kWarpKeys / 16; ++sub) {
            const int at = warp * kWarpKeys + sub * 16;  // first of 16 keys
            const int key0 = (u - it.first) * kKeys + at;
            if (key0 >= it.w.len) break;  // behind the last token
            const uint8_t* kc = ring + st * St::BYTES + at * VB;
            const uint8_t* vc = kc + St::CODES;
            const uint16_t* ks = reinterpret_cast<const uint16_t*>(ring + st * St::BYTES + 2 * St::CODES) + at * G;
            const uint16_t* vs = ks + St::STEPS / 2;

            // ---- scores of keys key0 + kr and key0 + kr + 8
            uint32_t ka[G], kb[G];
            float sa[G], sb[G];
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(kc + kr * VB + 16 * t);
                const uint4 y = *reinterpret_cast<const uint4*>(kc + (kr + 8) * VB + 16 * t);
                ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
                kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
                const uint2 p = *reinterpret_cast<const uint2*>(ks + kr * G);
                const uint2 q = *reinterpret_cast<const uint2*>(ks + (kr + 8) * G);
                sa[0] = __uint_as_float(p.x << 16), sa[1] = __uint_as_float(p.x & 0xffff0000u);
                sa[2] = __uint_as_float(p.y << 16), sa[3] = __uint_as_float(p.y & 0xffff0000u);
                sb[0] = __uint_as_float(q.x << 16), sb[1] = __uint_as_float(q.x & 0xffff0000u);
                sb[2] = __uint_as_float(q.y << 16), sb[3] = __uint_as_float(q.y & 0xffff0000u);
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(kc + kr * VB + 8 * t);
                const uint2 y = *reinterpret_cast<const uint2*>(kc + (kr + 8) * VB + 8 * t);
                ka[0] = x.x, ka[1] = x.y;
                kb[0] = y.x, kb[1] = y.y;
                const uint32_t p = *reinterpret_cast<const uint32_t*>(ks + kr * G);
                const uint32_t q = *reinterpret_cast<const uint32_t*>(ks + (kr + 8) * G);
                sa[0] = __uint_as_float(p << 16), sa[1] = __uint_as_float(p & 0xffff0000u);
                sb[0] = __uint_as_float(q << 16), sb[1] = __uint_as_float(q & 0xffff0000u);
            }
            float sv[NT][4];  // (key kr, col 0), (key kr, col 1), (key kr + 8, col 0), (key kr + 8, col 1)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sv[nt][0] = sv[nt][1] = sv[nt][2] = sv[nt][3] = 0.0f;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                const uint32_t a0 = raw_pair<0>(ka[gr]), a1 = raw_pair<0>(kb[gr]), a2 = raw_pair<1>(ka[gr]), a3 = raw_pair<1>(kb[gr]);
                const uint32_t b0 = raw_pair<2>(ka[gr]), b1 = raw_pair<2>(kb[gr]), b2 = raw_pair<3>(ka[gr]), b3 = raw_pair<3>(kb[gr]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float d[4];
                    mma_bf16_from(d, a0, a1, a2, a3, qf[nt][gr][0], qf[nt][gr][1], c0[nt][gr]);
                    mma_bf16(d, b0, b1, b2, b3, qf[nt][gr][2], qf[nt][gr][3]);
                    sv[nt][0] = fmaf(d[0], sa[gr], sv[nt][0]);
                    sv[nt][1] = fmaf(d[1], sa[gr], sv[nt][1]);
                    sv[nt][2] = fmaf(d[2], sb[gr], sv[nt][2]);
                    sv[nt][3] = fmaf(d[3], sb[gr], sv[nt][3]);
                }
            }
            const bool tail = key0 + 16 > least;  // some row does not see all of these keys
            if (tail) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (key0 + kr >= lim[nt][e]) sv[nt][e] = -INFINITY;
                        if (key0 + kr + 8 >= lim[nt][e]) sv[nt][2 + e] = -INFINITY;
                    }
            }
            // ---- maximum, raised rarely
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) raise |= fmaxf(sv[nt][e], sv[nt][2 + e]) > thr[nt][e];
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(sv[nt][e], sv[nt][2 + e]);
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = fmaxf(m, mx[nt][e]);
                        const float f = exp2_approx(mx[nt][e] == -INFINITY ? -INFINITY : in_units(mx[nt][e], sc[nt][e]) - in_units(m, sc[nt][e]));
                        mx[nt][e] = m;
                        ref[nt][e] = m == -INFINITY ? 0.0f : m;
                        thr[nt][e] = m + kRaise / sc[nt][e];
                        den[nt][e] *= f;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[nt][i][e] *= f;
                            o[nt][i][2 + e] *= f;
                        }
                    }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = exp2_approx((sv[nt][e] - ref[nt][e & 1]) * sc[nt][e & 1]);
                den[nt][0] += p[0] + p[2];
                den[nt][1] += p[1] + p[3];
                pf[nt][0] = transpose8x8(pack_bf16(p[0], p[1]));
                pf[nt][1] = transpose8x8(pack_bf16(p[2], p[3]));
            }

            // ---- values: score rows 2t, 2t + 1 (pair 0) and 2t + 8, 2t + 9 (pair 1)
            uint32_t s16[2][2], s24[2][2];  // [key pair][word]
            uint32_t xw[2][2][2];           // [key pair][word][nibbles 0-3 / 4-7]: the two keys' halves
#pragma unroll
            for (int kp = 0; kp < 2; ++kp) {
                const int k0 = 2 * t + (t & 1) + 8 * kp, k1 = 2 * t + 1 - (t & 1) + 8 * kp;  // the keys of these rows
                uint32_t st0, st1;  // steps of the two keys for this lane's words
                if constexpr (D == 128) {
                    st0 = *reinterpret_cast<const uint32_t*>(vs + k0 * G + ((2 * r) & 3));
                    st1 = *reinterpret_cast<const uint32_t*>(vs + k1 * G + ((2 * r) & 3));
                } else {
                    st0 = vs[k0 * G + (r & 1)];
                    st1 = vs[k1 * G + (r & 1)];
                }
                if (tail) {  // steps behind the last token are whatever the page holds
                    if (key0 + k0 >= it.w.len) st0 = 0;
                    if (key0 + k1 >= it.w.len) st1 = 0;
                }
                const uint32_t lo = __byte_perm(st0, st1, 0x5410);
                s16[kp][0] = bf16x2_mul(lo, kBf16x2Sixteen);
                s24[kp][0] = bf16x2_mul(lo, kBf16x2MinusTwentyFour);
                if constexpr (D == 128) {
                    const uint32_t hi = __byte_perm(st0, st1, 0x7632);
                    s16[kp][1] = bf16x2_mul(hi, kBf16x2Sixteen);
                    s24[kp][1] = bf16x2_mul(hi, kBf16x2MinusTwentyFour);
                    const uint2 x = *reinterpret_cast<const uint2*>(vc + k0 * VB + 8 * r);
                    const uint2 y = *reinterpret_cast<const uint2*>(vc + k1 * VB + 8 * r);
                    xw[kp][0][0] = __byte_perm(x.x, y.x, 0x5410);
                    xw[kp][0][1] = __byte_perm(x.x, y.x, 0x7632);
                    xw[kp][1][0] = __byte_perm(x.y, y.y, 0x5410);
                    xw[kp][1][1] = __byte_perm(x.y, y.y, 0x7632);
                } else {
                    const uint32_t x = *reinterpret_cast<const uint32_t*>(vc + k0 * VB + 4 * r);
                    const uint32_t y = *reinterpret_cast<const uint32_t*>(vc + k1 * VB + 4 * r);
                    xw[kp][0][0] = __byte_perm(x, y, 0x5410);
                    xw[kp][0][1] = __byte_perm(x, y, 0x7632);
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                // D = 128: rows r / r + 8 of tile i are nibble i of the lane's first / second word;
                // D = 64: nibbles i / i + 4 of its word
                uint32_t f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int kp = e >> 1, second = e & 1;
                    const int word = D == 128 ? second : 0;
                    const int nib = D == 128 ? i : i + 4 * second;
                    const uint32_t x = xw[kp][word][nib >> 2];
                    const uint32_t un = (nib & 3) == 0 ? kv4_unit_pair<0>(x) : (nib & 3) == 1 ? kv4_unit_pair<1>(x) : (nib & 3) == 2 ? kv4_unit_pair<2>(x) : kv4_unit_pair<3>(x);
                    f[e] = bf16x2_fma(un, s16[kp][word], s24[kp][word]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][i], f[0], f[1], f[2], f[3], pf[nt][0], pf[nt][1]);
            }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty(st));
        }
        if (!ok) {
            if (lane == 0) {
                atomicOr(a.err, kErrTimeout);
                *abort_flag = 1;
            }
            // fall through to the barriers below with what there is: the other warps meet there too
            u = u1;
        }

        // ---- join the four warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float d = den[nt][e];
                d += __shfl_xor_sync(0xffffffffu, d, 4);
                d += __shfl_xor_sync(0xffffffffu, d, 8);
                d += __shfl_xor_sync(0xffffffffu, d, 16);
                if (r == 0) {
                    stats[(warp * RB + nt * 8 + 2 * t + e) * 2] = mx[nt][e] == -INFINITY ? -INFINITY : in_units(mx[nt][e], sc[nt][e]);
                    stats[(warp * RB + nt * 8 + 2 * t + e) * 2 + 1] = d;
                }
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // dim of accumulator element e: word w of the vector, nibble n
                    const int second = e >> 1;
                    const int w = D == 128 ? 2 * r + second : r;
                    const int n = D == 128 ? i : i + 4 * second;
                    const int dim = 32 * (w % G) + 8 * (w / G) + n;
                    merge[(warp * RB + nt * 8 + 2 * t + (e & 1)) * D + dim] = o[nt][i][e];
                }
        // The producer may set the flag at any time, so the warps leave by what they brought to the barrier, which is the
        // same for all four: one that left while another went on to the next barrier would keep it there for good.
        if (consumers_meet(!ok || *abort_flag)) {
            join = make_int4(0, 0, 0, kGaveUp);
            break;
        }
        const bool starts = begin == it.first, ends = end == it.end;
        const bool whole = starts && ends;
        float* slot = a.slots + (size_t)(2 * c + (starts ? 1 : 0)) * RB * (D + 2);
        for (int x = tid; x < rows * (D / 4); x += 32 * kWarps) {
            const int row = x / (D / 4), d4 = 4 * (x % (D / 4));
            float m = -INFINITY, den_all = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stats[(w * RB + row) * 2]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = stats[(w * RB + row) * 2];
                const float f = mw == -INFINITY ? 0.0f : exp2_approx(mw - m);
                const float4 ov = *reinterpret_cast<const float4*>(merge + (w * RB + row) * D + d4);
                den_all += f * stats[(w * RB + row) * 2 + 1];
                v.x += f * ov.x, v.y += f * ov.y, v.z += f * ov.z, v.w += f * ov.w;
            }
            // a warp that saw only NaN scores has no maximum but a NaN denominator
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (stats[(w * RB + row) * 2 + 1] != stats[(w * RB + row) * 2 + 1]) den_all = NAN;
            if (whole) {
                const int ri = it.rb * RB + row;
                const float inv = den_all == 0.0f ? 0.0f : 1.0f / den_all;
                uint16_t* op = a.out + (int64_t)(it.w.row0 + ri / a.group) * a.out_stride + (it.head * a.group + ri % a.group) * D + d4;
                *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            } else {
                float* sp = slot + row * (D + 2);
                *reinterpret_cast<float2*>(sp + d4) = make_float2(v.x, v.y);
                *reinterpret_cast<float2*>(sp + d4 + 2) = make_float2(v.z, v.w);
                if (d4 == 0) *reinterpret_cast<float2*>(sp + D) = make_float2(m, den_all);
            }
        }
        if (starts && !ends) {
            // this CTA holds the item's first piece: the last one is with the CTA of its last unit
            const int last = (int)(((long long)it.end * ctas + total - 1) / total) - 1;
            join = make_int4(it.w.row0, it.head, it.rb | (rows << 24), last);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    }
    if (tid == 0) a.joins[c] = join;
}

// Join the pieces of split items: block c takes the item whose first piece CTA c
// held: slot 2c + 1, then slot 2c' of the CTAs c' up to the one that held its last
// unit, in order. A warp takes a row: its lanes first read the pieces' maxima, then the
// denominators and the sums, 16 bytes each (D = 64: two pieces at once), eight loads in
// flight. With more warps than rows a row's pieces are shared by several, which meet in
// shared memory: 89 pieces of 4 rows 28.0 -> 25.0 us with the units' kernel, 32 pieces
// 10.5 -> 9.9. For items of few pieces the larger blocks cost more than that gives
// (64 sequences 57.3 -> 58.4).
template <int D, int RB, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) kv4_join_kernel(const RowsArgs a) {
    constexpr int VL = D / 4;        // lanes of a row
    constexpr int PP = 32 / VL;      // pieces at once
    __shared__ float4 part[WARPS][VL];
    __shared__ float part_den[WARPS];
    grid_dependency_wait();
    grid_dependents_launch();
    const int4 j = a.joins[blockIdx.x];
    if (j.w < 0) return;
    const int rows = j.z >> 24;
    int share = 1;  // warps of a row
    if (WARPS > RB)
        while (2 * share * rows <= WARPS) share *= 2;
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = warp / share, turn = warp % share;
    const int pieces = j.w - c + 1;
    auto slot = [&](int p) { return a.slots + ((size_t)(2 * (c + p) + (p == 0 ? 1 : 0)) * RB + row) * (D + 2); };
    const int sub = lane / VL, d4 = 4 * (lane % VL);
    float den = 0.0f;
    bool lost = false;  // a piece is missing: the row is left as it was
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows) {
        float m = -INFINITY;
#pragma unroll 4
        for (int p = lane; p < pieces; p += 32) {
            m = fmaxf(m, slot(p)[D]);
            lost |= a.joins[c + p].w == kGaveUp;
        }
        m = warp_max(m);
        lost = __any_sync(0xffffffffu, lost);
        constexpr int BATCH = 8 * PP;  // pieces in flight
        for (int p0 = turn * BATCH; p0 < pieces; p0 += share * BATCH) {
            float4 x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {  // past the end: the last piece, not added
                const float* sp = slot(min(p0 + q * PP + sub, pieces - 1)) + d4;  // 8-byte aligned
                const float2 lo = *reinterpret_cast<const float2*>(sp), hi = *reinterpret_cast<const float2*>(sp + 2);
                x[q] = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
            float f = 0.0f, d = 0.0f;
            if (lane < BATCH && p0 + lane < pieces) {
                const float2 st = *reinterpret_cast<const float2*>(slot(p0 + lane) + D);
                f = st.x == -INFINITY ? (st.y != st.y ? 1.0f : 0.0f) : exp2_approx(st.x - m);
                d = f * st.y;
            }
            den += warp_sum(d);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float g = __shfl_sync(0xffffffffu, f, q * PP + sub);
                if (p0 + q * PP + sub < pieces) v.x += g * x[q].x, v.y += g * x[q].y, v.z += g * x[q].z, v.w += g * x[q].w;
            }
        }
        if (PP == 2) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, 16), v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
            v.z += __shfl_xor_sync(0xffffffffu, v.z, 16), v.w += __shfl_xor_sync(0xffffffffu, v.w, 16);
        }
        if (turn && sub == 0) {
            part[warp][lane] = v;
            if (lane == 0) part_den[warp] = den;
        }
    }
    if (share > 1) __syncthreads();  // the same for the whole block
    if (turn || sub || row >= rows || lost) return;
    for (int w = warp + 1; w < warp + share; ++w) {
        const float4 o = part[w][lane];
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        den += part_den[w];
    }
    const float inv = den == 0.0f ? 0.0f : 1.0f / den;
    const int ri = (j.z & 0xffffff) * RB + row;
    *reinterpret_cast<uint2*>(a.out + (int64_t)(j.x + ri / a.group) * a.out_stride + (j.y * a.group + ri % a.group) * D + d4) =
        make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
}

template <int D, int NT>
cudaError_t launch_rows(const RowsArgs& args, int ctas_cap, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static int resident[64];  // CTAs the device holds at once with a small batch
    const size_t smem = RowsSmem<D, NT>::bytes(args.batch.S);
    auto kern = kv4_rows_kernel<D, NT>;
    if (dev >= 64 || !resident[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RowsSmem<D, NT>::bytes(kKv4MaxSeqs));
        if (e != cudaSuccess) return e;
        int sms = 0, per = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, kThreads, RowsSmem<D, NT>::bytes(64));
        if (e != cudaSuccess) return e;
        if (dev < 64) resident[dev] = sms * per;
    }
    const int grid = min(ctas_cap, dev < 64 ? resident[dev] : 148);
    e = launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), smem, s, args);
    if (e != cudaSuccess) return e;
    constexpr int RB = 8 * NT;
    // pieces of an item, should the lengths be alike
    if (RB == 8 && grid >= 8 * (int64_t)args.batch.S * args.cache.hkv)
        return launch_pdl(kv4_join_kernel<D, RB, 16>, dim3((unsigned)grid), dim3(32 * 16), 0, s, args);
    return launch_pdl(kv4_join_kernel<D, RB, RB>, dim3((unsigned)grid), dim3(32 * RB), 0, s, args);
}

}  // namespace

namespace {
// Rows that share a key/value head up to which the decode kernel runs (two n-tiles of the MMA, all it holds). Tiles
// instead: 64 x 2048 keys with 16 rows 93 us (here 55), 8 x 600 keys with 15 rows 18.8 (13.8), 1 x 8192 keys with 5
// rows 32 (14.6).
constexpr int64_t kRowsMax = 16;

inline bool by_tiles(int64_t max_q, int64_t group) { return max_q * group > kRowsMax; }

// Slots of pieces, then the joins.
size_t rows_slots_bytes(int D) { return (size_t)2 * kMaxCtas * 16 * (D + 2) * 4; }
}  // namespace

size_t kv4_attention_workspace_bytes(int64_t max_q, int64_t group, int D) {
    return by_tiles(max_q, group) ? kv4_tile_workspace_bytes(D) : rows_slots_bytes(D) + (size_t)kMaxCtas * sizeof(int4);
}

cudaError_t launch_kv4_attention(const uint16_t* q, int64_t q_stride, int64_t M, int Hq, int D, int64_t max_q, float scale,
                                 const Kv4View& cache, const Kv4Seqs& batch, uint16_t* out, int64_t out_stride, void* ws,
                                 cudaStream_t s) {
    if (by_tiles(max_q, Hq / cache.hkv))
        return launch_kv4_tile(q, q_stride, M, Hq, D, max_q, scale, cache, batch, out, out_stride, ws, s);
    RowsArgs a;
    a.q = q, a.out = out, a.q_stride = q_stride, a.out_stride = out_stride;
    a.cache = cache, a.batch = batch;
    a.M = (int)M, a.group = Hq / cache.hkv, a.max_q = (int)std::min<int64_t>(max_q, M);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.least_shift = std::max(10, kSpacing - 127 + 1 + std::ilogb(a.scale_log2) + 1);
    a.slots = (float*)ws;
    a.joins = (int4*)((char*)ws + rows_slots_bytes(D));
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    const bool two = (int64_t)a.group * a.max_q > 8;
    if (D == 128) return two ? launch_rows<128, 2>(a, kMaxCtas, s) : launch_rows<128, 1>(a, kMaxCtas, s);
    return two ? launch_rows<64, 2>(a, kMaxCtas, s) : launch_rows<64, 1>(a, kMaxCtas, s);
}

}  // namespace bl
