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
//                        row's exponentials of a block sum up to more than 2^10.
// Work split as in kv4_attn.cu: the units of all items in one line, an equal
// contiguous range per CTA (one CTA per SM), pieces of split items joined by a
// second kernel in a fixed order. Causal limits cut an item's blocks short.
//
// The weights are rounded to bf16 for the product with the values; the denominator sums
// them as they are.
//
// Measured (20 query, 5 key/value heads of 128): 2047 tokens on 30001 keys 528 us in a
// burst, 1150 TFLOP/s, 596 sustained, 1019; the tensor pipe 53% busy, special functions
// 40%, issue slots 57%. Six prompts of 100 to 4096 tokens 186 us, a third of it the starts
// and ends of items. No pipe is full: timing copies at 2048 tokens on 16384 keys took 291
// us whole, 209 without the softmax, 265 with one MMA of eight, 179 with neither, so the
// larger part is unpacking and the hand-overs between the roles. Pieces of one tile take
// as long a block as two; letting both warpgroups share the blocks of one gained 3% there
// and cost 8% elsewhere.
//
// Every wait is bounded (1 s); one that gives up sets the device error word,
// lets the CTA drain and returns.
#include <algorithm>
#include <type_traits>

#include <cfloat>

#include "kv4.cuh"
#include "tc_ptx.cuh"

namespace bl {
namespace {

constexpr int BLK = 128;          // keys per unit
constexpr int TM = 128;           // rows per tile
constexpr int ROWS = 2 * TM;      // rows per item
constexpr int KV_STAGES = 4;      // unpacked tiles: K, V, K, V
constexpr int CODE_STAGES = 3;    // packed tiles
constexpr int SOFT_WARPS = 8;     // two tiles x four warps
constexpr int UNPACK_WARPS = 8;
constexpr int LOAD_WARP = SOFT_WARPS + UNPACK_WARPS, MMA_WARP = LOAD_WARP + 1;
constexpr int THREADS = 32 * (LOAD_WARP + 4);
// registers a thread, per warpgroup: two of softmax, two of unpacking, one of the rest (launched with 96)
constexpr int LAUNCH_REGS = 96, SOFT_REGS = 160, UNPACK_REGS = 48, REST_REGS = 56;
static_assert(2 * SOFT_REGS + 2 * UNPACK_REGS + REST_REGS <= 5 * LAUNCH_REGS && THREADS * LAUNCH_REGS <= 65536, "register split");
constexpr int MAX_CTAS = 148;     // sizes the workspace
// What starting and ending an item costs, in units (it evens out the ranges): 4096 tokens of one prompt 115 us with 4,
// 137 with 2, 122 with 8; 8 prompts of 512 47 with 4, 51 with 2, 43 with 8.
constexpr int ITEM_UNITS = 4;
constexpr int SEQ_GROUP = 32;     // sequences per entry of the coarse unit table
constexpr uint64_t WAIT_NS = 1000000000ull;
constexpr int GAVE_UP = -2;
constexpr float FAR = 16777216.0f;    // scaled maximum whose rounding is one in the exponent
constexpr float RAISE_SUM = 1024.0f;  // sum of a row's exponentials over a block that raises its maximum

struct TileArgs {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    Kv4View cache;
    Kv4Seqs batch;
    int M, group, max_q;
    uint64_t group_inv;  // ceil(2^40 / group): rows / group as a multiplication
    float scale_log2;
    float* slots;   // [2 gridDim.x] pieces: [D / 4][ROWS] float4 sums, then [ROWS] (maximum, denominator)
    int4* joins;    // [gridDim.x] item whose first piece the CTA holds: first row, head, item | rows << 20, last CTA;
                    // .w = -1: none, GAVE_UP: none, and its own pieces are not all there
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

// Low word of a shared-memory matrix descriptor (address and leading offset in
// 16-byte units); the high word is the same for every operand here: 1024 bytes
// between groups of 8 rows, version 1, 128-byte swizzle.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
    return ((saddr & 0x3FFFFu) >> 4) | ((lbo_bytes >> 4) << 16);
}
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// bf16 inputs, fp32 accumulators; A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(DESC_HI)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(idesc), "r"(acc), "r"(DESC_HI)
        : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// 2^x of two values on the multiply-add pipe, for a share of the exponentials
// (the special-function pipe alone would take as long as the MMAs): x = n + f,
// |f| <= 1/2, by adding 1.5 * 2^23 + 128; 2^f by a cubic (fitted to the least
// largest relative error, 7.5e-05, a fraction of a bf16 rounding); 2^n as an
// exponent. x below -127 gives 0, a NaN stays one. An x of 128 or more gives
// nonsense: its sum t is no longer POLY_MAGIC plus a byte; `seen`, all sums' bits,
// shows it (half an instruction a value; a clamp from above, or a maximum of the
// arguments, made the prompts 3% slower).
constexpr uint32_t POLY_MAGIC = 0x4B400000u;  // 1.5 * 2^23
constexpr int POLY_EVERY = 4;
__device__ __forceinline__ float2 exp2_poly(float2 x, uint32_t& seen) {
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.x));
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.y));
    const float2 magic = make_float2(12583040.0f, 12583040.0f), minus = make_float2(-12583040.0f, -12583040.0f);
    const float2 t = add2(x, magic);
    seen |= __float_as_uint(t.x) | __float_as_uint(t.y);
    const float2 n = add2(t, minus);
    const float2 f = fma2(n, make_float2(-1.0f, -1.0f), x);
    float2 y = fma2(f, make_float2(0.0551713221f, 0.0551713221f), make_float2(0.242610544f, 0.242610544f));
    y = fma2(y, f, make_float2(0.693260968f, 0.693260968f));
    y = fma2(y, f, make_float2(0.999928117f, 0.999928117f));
    y.x *= __uint_as_float((__float_as_uint(t.x) << 23) - 0x00800000u);
    y.y *= __uint_as_float((__float_as_uint(t.y) << 23) - 0x00800000u);
    return y;
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

// n / group for 0 <= n < 2^29 (group <= 1024): exact, since n * group < 2^40.
__device__ __forceinline__ int per_group(const TileArgs& a, int n) { return (int)(((uint64_t)n * a.group_inv) >> 40); }

// Blocks of item t of a sequence: up to the last key that its last row sees.
__device__ __forceinline__ int blocks_of(const TileArgs& a, const Seq& w, int t) {
    const int last = min(w.n_q - 1, per_group(a, (t + 1) * ROWS - 1));
    return max(1, (w.len - w.n_q + last + 1 + BLK - 1) / BLK);
}

__device__ __forceinline__ int warp_scan(int v) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// Whether q_start decreases at a sequence of group g. The host bounds the units by 2^31 from M rows in all; seq_of
// checks a sequence for itself, but only sequences in order have rows of their own, which add up to M.
__device__ __forceinline__ bool group_decreases(const TileArgs& a, int g) {
    const int s = g * SEQ_GROUP + (int)(threadIdx.x & 31);
    return __any_sync(0xffffffffu, s < a.batch.S && a.batch.q_start[s] > a.batch.q_start[s + 1]);
}

// Units of the SEQ_GROUP sequences of group g, sequence g * SEQ_GROUP + lane in each lane; the warp shares the
// tiles of each long sequence.
__device__ __forceinline__ int group_units(const TileArgs& a, int g, bool report) {
    const int lane = threadIdx.x & 31, s = g * SEQ_GROUP + lane;
    Seq w;
    w.row0 = w.n_q = w.len = w.tiles = 0;
    if (s < a.batch.S) w = seq_of(a, s, report);
    int n = 0;
    if (w.tiles <= 2) {
        for (int t = 0; t < w.tiles; ++t) n += ITEM_UNITS + blocks_of(a, w, t);
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, w.tiles > 2); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1;
        Seq x;
        x.n_q = __shfl_sync(0xffffffffu, w.n_q, from);
        x.len = __shfl_sync(0xffffffffu, w.len, from);
        x.tiles = __shfl_sync(0xffffffffu, w.tiles, from);
        int sum = 0;
        for (int t = lane; t < x.tiles; t += 32) sum += ITEM_UNITS + blocks_of(a, x, t);
        sum = warp_sum(sum);
        if (lane == from) n = sum;
    }
    return n * a.cache.hkv;
}

// The pieces of this CTA's range, in order; every role walks its own copy.
struct Pieces {
    int u, u1;                      // next unit, end of the range
    int s, t, head, first, blocks;  // current item, its first unit
    Seq w;

    // An item spans ITEM_UNITS, then its blocks; a range that holds none of its blocks has no piece of it.
    __device__ bool next(const TileArgs& a, int& b0, int& b1) {
        while (u < u1) {
            while (u >= end()) {  // move to the item that holds u
                first = end();
                if (++head == a.cache.hkv) {
                    head = 0;
                    if (++t >= w.tiles) {
                        t = 0;
                        do {
                            w = seq_of(a, ++s, false);
                        } while (w.tiles == 0);  // a later sequence has units: u < u1 <= total, and total is exact
                    }
                }
                blocks = blocks_of(a, w, t);
            }
            b0 = max(0, u - first - ITEM_UNITS);
            b1 = min(blocks, u1 - first - ITEM_UNITS);
            u = min(u1, end());
            if (b1 > b0) return true;
        }
        return false;
    }

    __device__ int end() const { return first + ITEM_UNITS + blocks; }
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
    __shared__ int coarse[kKv4MaxSeqs / SEQ_GROUP + 1];  // [g + 1]: units up to the end of group g of sequences
    __shared__ Pieces start_sh;
    __shared__ int total_sh;
    __shared__ int valid_sh[CODE_STAGES];  // keys of a packed tile, -1 after the last

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
        for (int i = 0; i < KV_STAGES; ++i) tc::mbar_init(tfull(i), 32 * UNPACK_WARPS), tc::mbar_init(tempty(i), 1);
        for (int i = 0; i < CODE_STAGES; ++i) tc::mbar_init(cfull(i), 1), tc::mbar_init(cempty(i), 32 * UNPACK_WARPS);
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

    // ---- units of all sequences, and where this CTA's range of them starts
    const int groups = (a.batch.S + SEQ_GROUP - 1) / SEQ_GROUP;
    for (int g = warp; g < groups; g += THREADS / 32) {
        const bool decreases = group_decreases(a, g);
        const int sum = decreases ? -1 : warp_sum(group_units(a, g, blockIdx.x == 0));
        if (lane == 0) {
            coarse[g + 1] = sum;
            if (decreases && blockIdx.x == 0) atomicOr(a.err, kErrBadBatch);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int g = g0 + lane;
            const int own = g < groups ? coarse[g + 1] : 0;
            if (__any_sync(0xffffffffu, own < 0)) {  // a batch out of order has no work; up to here its sums are sound
                carry = 0;
                break;
            }
            const int sum = carry + warp_scan(own);
            if (g < groups) coarse[g + 1] = sum;
            carry = __shfl_sync(0xffffffffu, sum, 31);
        }
        __syncwarp();
        const int ctas = min((int)gridDim.x, carry);
        if ((int)blockIdx.x < ctas) {
            Pieces p;
            p.u = (int)((long long)carry * blockIdx.x / ctas);
            p.u1 = (int)((long long)carry * (blockIdx.x + 1) / ctas);
            int g = 0;  // the group that holds u: the number of groups that end at or before it
            for (int g0 = 0; g0 < groups; g0 += 32)
                g += __popc(__ballot_sync(0xffffffffu, g0 + lane < groups && coarse[g0 + lane + 1] <= p.u));
            const int n = group_units(a, g, false);
            const int before = g ? coarse[g] : 0;
            const int upto = before + warp_scan(n);
            const int in = __popc(__ballot_sync(0xffffffffu, upto <= p.u));  // < 32: the group holds u
            p.s = g * SEQ_GROUP + in;
            p.w = seq_of(a, p.s, false);
            int at = __shfl_sync(0xffffffffu, upto - n, in);  // units before the sequence
            for (int t0 = 0;; t0 += 32) {
                const int t = t0 + lane;
                const int b = t < p.w.tiles ? (ITEM_UNITS + blocks_of(a, p.w, t)) * a.cache.hkv : 0;
                const int end = at + warp_scan(b);
                const int k = __popc(__ballot_sync(0xffffffffu, t < p.w.tiles && end <= p.u));
                if (k < 32) {
                    p.t = t0 + k;
                    at = __shfl_sync(0xffffffffu, end - b, k);
                    break;
                }
                at = __shfl_sync(0xffffffffu, end, 31);
            }
            p.blocks = blocks_of(a, p.w, p.t);
            p.head = (p.u - at) / (ITEM_UNITS + p.blocks);
            p.first = at + p.head * (ITEM_UNITS + p.blocks);
            if (lane == 0) start_sh = p;
        }
        if (lane == 0) total_sh = carry;
    }
    __syncthreads();
    const int total = total_sh;
    const int ctas = min((int)gridDim.x, total);
    const int c = blockIdx.x;
    if (c >= ctas) {
        if (tid == 0) a.joins[c] = make_int4(0, 0, 0, -1);
        return;
    }
    if (warp == MMA_WARP) {
        tc::tmem_alloc(tc::smem_u32(&tmem_base_sh), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base_sh;
    // TMEM columns: scores of tile i at 128 i (P over their first half), sums of tile i at 256 + D i
    auto give_up = [&]() {
        atomicOr(a.err, kErrTimeout);
        *aborted = 1;
    };

    if (warp >= LOAD_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REST_REGS));
        if (warp == LOAD_WARP) {
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
                        if (lane == 0) valid_sh[st] = max(0, p.w.len - b * BLK);
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
            bool told = false;
            if (ok) {  // tell the unpackers that this was all
                const int st = g % CODE_STAGES;
                if (g >= CODE_STAGES) ok = tc::mbar_wait(cempty(st), (g / CODE_STAGES - 1) & 1, WAIT_NS);
                ok = __all_sync(0xffffffffu, ok);
                if (ok && lane == 0) {
                    valid_sh[st] = -1;
                    tc::mbar_arrive(cfull(st));
                    told = true;
                }
            }
            if (lane == 0) {
                if (!ok) give_up();
                // Let the copies still in flight land before the CTA exits: the unpackers wait for them too, unless they
                // give up. The stage whose barrier told them the end was empty, so its copies have landed.
                for (uint32_t h = g >= CODE_STAGES ? g - CODE_STAGES + (told ? 1 : 0) : 0; h < g; ++h)
                    tc::mbar_wait(cfull(h % CODE_STAGES), (h / CODE_STAGES) & 1, WAIT_NS);
            }
        } else if (warp == MMA_WARP) {
            // ------------------------------------------------------------ MMA issuer: one elected lane. (A warp that
            // walks along is 2% slower and must vote after every wait: a lane that falls behind misses a phase.)
            if (elect_one()) {
                constexpr uint32_t id_s = idesc_bf16(TM, BLK, false);
                constexpr uint32_t id_o = idesc_bf16(TM, D, true);
                Pieces p = start_sh;
                uint32_t n = 0;                // blocks so far (K tile 2n, V tile 2n + 1 of the ring)
                uint32_t np0 = 0, np1 = 0;     // P tiles consumed
                uint32_t nq0 = 0, nq1 = 0;     // Q tiles consumed
                const uint32_t q_lo = desc_lo(tc::smem_u32(sQ), 16);
                const uint32_t k_lo = desc_lo(tc::smem_u32(sT), 16), v_lo = desc_lo(tc::smem_u32(sT), C::HALF);
                int b0, b1;
                bool ok = true;
                auto wait = [&](uint32_t b, uint32_t parity) {
                    ok = tc::mbar_wait(b, parity, WAIT_NS);
                    tc::fence_after_sync();
                    return ok;
                };
                auto commit = [&](uint32_t b) { tc::mma_commit(b); };
                // `st` 0 / 1: the half of the ring (K tile 2 st, V tile 2 st + 1), a constant so that descriptors are too
                auto scores = [&](auto tile, auto st) {
                    constexpr int i = decltype(tile)::value, o = 2 * decltype(st)::value * (C::TILE >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k / 4) * C::HALF + (k % 4) * 32) >> 4;
                        mma_ss(tmem + 128 * i, q_lo + i * (C::TILE >> 4) + off, k_lo + o + off, id_s, k != 0);
                    }
                    tc::mma_commit(sfull(i));
                };
                auto values = [&](auto tile, auto st, bool first) {
                    constexpr int i = decltype(tile)::value, o = (2 * decltype(st)::value + 1) * (C::TILE >> 4);
#pragma unroll
                    for (int k = 0; k < BLK / 16; ++k)
                        mma_ts(tmem + 256 + i * D, tmem + 128 * i + 8 * k, v_lo + o + ((k * 16 * 128) >> 4), id_o, k != 0 || !first);
                };
                using T0 = std::integral_constant<int, 0>;
                using T1 = std::integral_constant<int, 1>;
                // scores of an item's first block (block n of this CTA, in half `st` of the ring)
                auto open = [&](auto st, bool two) {
                    constexpr int h = decltype(st)::value;
                    if (!wait(tfull(2 * h), (n >> 1) & 1) || !wait(qfull(0), nq0++ & 1)) return false;
                    scores(T0{}, st);
                    if (two) {
                        if (!wait(qfull(1), nq1++ & 1)) return false;
                        scores(T1{}, st);
                    }
                    commit(tempty(2 * h));
                    return true;
                };
                // values of block n, scores of block n + 1 if the piece has it: tile 0, then tile 1
                auto step = [&](auto st, bool two, bool first, bool more) {
                    constexpr int h = decltype(st)::value;
                    using Next = std::integral_constant<int, 1 - h>;
                    if (!wait(tfull(2 * h + 1), (n >> 1) & 1)) return false;
                    if (more && !wait(tfull(2 * (1 - h)), ((n + 1) >> 1) & 1)) return false;
                    if (!wait(pfull(0), np0++ & 1)) return false;
                    values(T0{}, st, first);
                    if (more)
                        scores(T0{}, Next{});
                    else
                        commit(ofull(0));
                    if (two) {
                        if (!wait(pfull(1), np1++ & 1)) return false;
                        values(T1{}, st, first);
                        if (!more) commit(ofull(1));
                    }
                    commit(tempty(2 * h + 1));
                    if (more) {
                        if (two) scores(T1{}, Next{});
                        commit(tempty(2 * (1 - h)));
                    }
                    ++n;
                    return true;
                };
                while (ok && p.next(a, b0, b1)) {
                    const bool two = p.w.n_q * a.group - p.t * ROWS > TM;
                    if (!(n & 1 ? open(T1{}, two) : open(T0{}, two))) break;
                    for (int j = b0; j < b1; ++j)
                        if (!(n & 1 ? step(T1{}, two, j == b0, j + 1 < b1) : step(T0{}, two, j == b0, j + 1 < b1))) break;
                }
                if (!ok) give_up();
            }
            __syncwarp();
        }
    } else if (warp >= SOFT_WARPS) {
        // ---------------------------------------------------------------- unpack
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(UNPACK_REGS));
        // A lane owns the group `gr` of a key: four words and one step. The order in which lanes take the
        // octets makes both the word loads (32 lanes, 32 banks) and the 16-byte stores (8 lanes of a phase, 8
        // chunks of a 128-byte row) free of bank conflicts.
        constexpr int KPW = 32 / G;               // keys per warp and pass
        constexpr int KPP = UNPACK_WARPS * KPW;   // keys per pass
        constexpr int PASSES = BLK / KPP;
        const int gr = lane % G;
        const int row = (warp - SOFT_WARPS) * KPW + lane / G;  // key of the first pass
        int loads[4], stores[4];                  // byte offsets of the i-th octet, the same in every pass
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = D == 128 ? ((i + (row >> 1)) & 3) ^ (2 * (gr >> 1)) : (i + (row >> 2)) & 3;
            loads[i] = row * VB + 4 * (t * G + gr);
            stores[i] = (gr >> 1) * C::HALF + row * 128 + (((4 * (gr & 1) + t) ^ (row & 7)) << 4);
        }
        for (uint32_t g = 0;; ++g) {
            const int cs = g % CODE_STAGES, ts = g % KV_STAGES;
            if (*aborted || !tc::mbar_wait(cfull(cs), (g / CODE_STAGES) & 1, WAIT_NS) ||
                (g >= KV_STAGES && valid_sh[cs] >= 0 && !tc::mbar_wait(tempty(ts), (g / KV_STAGES - 1) & 1, WAIT_NS))) {
                give_up();
                break;
            }
            const int valid = valid_sh[cs];
            if (valid < 0) break;
            const uint8_t* codes = sC + cs * C::PACKED;
            uint8_t* tile = sT + ts * C::TILE;
            // all loads first: the compiler may not move one across a store to shared memory
            uint32_t word[PASSES][4], st[PASSES];
#pragma unroll
            for (int pass = 0; pass < PASSES; ++pass) {
                st[pass] = *reinterpret_cast<const uint16_t*>(codes + C::CODES + (pass * KPP + row) * 2 * G + 2 * gr);
#pragma unroll
                for (int i = 0; i < 4; ++i) word[pass][i] = *reinterpret_cast<const uint32_t*>(codes + loads[i] + pass * KPP * VB);
            }
#pragma unroll
            for (int pass = 0; pass < PASSES; ++pass) {
                if (pass * KPP + row >= valid) st[pass] = 0;  // behind the last token: whatever the page holds
                st[pass] = __byte_perm(st[pass], 0, 0x1010);
                const uint32_t s16 = bf16x2_mul(st[pass], kBf16x2Sixteen), s24 = bf16x2_mul(st[pass], kBf16x2MinusTwentyFour);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = word[pass][i];
                    *reinterpret_cast<uint4*>(tile + stores[i] + pass * KPP * 128) =
                        make_uint4(bf16x2_fma(kv4_unit_pair<0>(x), s16, s24), bf16x2_fma(kv4_unit_pair<1>(x), s16, s24),
                                   bf16x2_fma(kv4_unit_pair<2>(x), s16, s24), bf16x2_fma(kv4_unit_pair<3>(x), s16, s24));
                }
            }
            tc::mbar_arrive(cempty(cs));
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(tfull(ts));
        }
    } else {
        // ---------------------------------------------------------------- softmax: tile i, row r of it
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFT_REGS));
        const int i = warp >> 2, r = tid & (TM - 1);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + 128 * i + lanes, tO = tmem + 256 + D * i + lanes;
        const float sc = a.scale_log2;
        Pieces p = start_sh;
        uint32_t ns = 0, no = 0;
        int4 join = make_int4(0, 0, 0, -1);
        constexpr int LPR = D / 8, RPI = 32 / LPR, QN = 32 / RPI;  // lanes of a row, rows and count of 16-byte accesses
        const int oct = lane % LPR;
        // The next piece that has rows in this tile: what the thread needs to know of it. Its queries start on their
        // way to L2; they are loaded once the tile's memory is free.
        int b0 = 0, b1 = 0, limit = 0, least = 0;
        int64_t row_out = -1, row_q = -1;  // this row's offsets in out and q, -1 for a row that does not exist
        bool starts = false, ends = false;
        auto fetch = [&]() {
            int rows;
            do {
                if (!p.next(a, b0, b1)) return false;
                rows = min(ROWS, p.w.n_q * a.group - p.t * ROWS);
                starts = b0 == 0, ends = b1 == p.blocks;
                if (starts && !ends) {
                    const int last = (int)(((long long)p.end() * ctas + total - 1) / total) - 1;
                    join = make_int4(p.w.row0, p.head, p.t | (rows << 20), last);
                }
            } while (i * TM >= rows);
            const bool live = i * TM + r < rows;
            const int ri = p.t * ROWS + i * TM + r;  // row of the sequence
            const int token = per_group(a, ri), qh = p.head * a.group + ri - token * a.group;
            limit = live ? min(p.w.len, p.w.len - p.w.n_q + token + 1) : 0;
            least = p.w.len - p.w.n_q + per_group(a, p.t * ROWS + i * TM) + 1;  // keys all rows see
            row_out = live ? (int64_t)(p.w.row0 + token) * a.out_stride + qh * D : -1;
            row_q = live ? (int64_t)(p.w.row0 + token) * a.q_stride + qh * D : -1;
            if (live) {
#pragma unroll
                for (int x = 0; x < D; x += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + row_q + x));
            }
            return true;
        };
        // 16 bytes `o8` of row `rr` of the tile's query memory
        auto cell = [&](int rr, int o8) {
            return reinterpret_cast<uint4*>(sQ + i * C::TILE + (o8 >> 3) * C::HALF + rr * 128 + (((o8 & 7) ^ (rr & 7)) << 4));
        };
        bool ok = true;
        bool have = fetch();
        while (have) {
            // the warp's 32 rows of queries, D / 8 lanes to a row
#pragma unroll 1
            for (int x0 = 0; x0 < QN; x0 += QN / 2) {
                uint4 v[QN / 2];
#pragma unroll
                for (int x = 0; x < QN / 2; ++x) {
                    const int64_t off = __shfl_sync(0xffffffffu, row_q, (x0 + x) * RPI + lane / LPR);
                    v[x] = make_uint4(0, 0, 0, 0);
                    if (off >= 0) v[x] = *reinterpret_cast<const uint4*>(a.q + off + 8 * oct);
                }
#pragma unroll
                for (int x = 0; x < QN / 2; ++x)
                    *cell((warp & 3) * 32 + (x0 + x) * RPI + lane / LPR, oct) =
                        make_uint4(__byte_perm(v[x].x, v[x].z, 0x5410), __byte_perm(v[x].x, v[x].z, 0x7632),
                                   __byte_perm(v[x].y, v[x].w, 0x5410), __byte_perm(v[x].y, v[x].w, 0x7632));
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(qfull(i));
            float mx = -INFINITY, msc = 0.0f, den = 0.0f;
            bool some_far = false;  // of the warp's rows
            for (int b = b0; b < b1; ++b, ++ns) {
                ok = !*aborted && tc::mbar_wait(sfull(i), ns & 1, WAIT_NS);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after_sync();
                const int seen = limit - b * BLK;  // columns this row sees
                const bool masked = b * BLK + BLK > least;
                uint32_t s[2][32];
                auto load = [&](int k) { tc::tmem_ld_32x32(tS + 32 * k, s[k & 1]); };
                auto mask = [&](int k) {
                    if (masked) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (32 * k + x >= seen) s[k & 1][x] = 0xFF800000u;
                    }
                };
                // Exponentials against the maximum so far. A row whose sum shows that its maximum has grown too much
                // (always on the first block, and while no score was above -inf) has it raised, and the warp takes the
                // pass again: the scores stay where they are until P is stored over them. Nothing else looks at the
                // scores' maximum.
                float sum = 0.0f;
                uint32_t pk[2][32];
                // A row whose scaled maximum is far from zero has the maximum itself taken off its scores, once it holds for
                // the block: the rounding of the scaled one, which the multiply-add leaves in every exponent, would pass the
                // exponent's range from 2^31 on.
                for (bool again = b == b0 || some_far;;) {
                    if (again) {
                        float m = -INFINITY;
                        load(0);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            tc::tmem_ld_wait();
                            if (k < 3) load(k + 1);
                            mask(k);
#pragma unroll
                            for (int x = 0; x < 32; x += 2)
                                m = max3(m, __uint_as_float(s[k & 1][x]), __uint_as_float(s[k & 1][x + 1]));
                        }
                        float f = 1.0f;
                        if (m > mx) {
                            const float now = fmaxf(m * sc, -FLT_MAX);  // a score below fp32 weighs nothing, but is no NaN
                            f = mx == -INFINITY ? 0.0f : exp2_approx(msc - now);
                            mx = m;
                            msc = now;
                            den = now > FLT_MAX ? NAN : den * f;  // above fp32: no softmax
                        }
                        some_far = __any_sync(0xffffffffu, fabsf(msc) >= FAR);
                        if (some_far) {
                            const float take = fabsf(msc) >= FAR ? mx : 0.0f;
#pragma unroll 1
                            for (int k = 0; k < 4; ++k) {
                                tc::tmem_ld_32x32(tS + 32 * k, s[0]);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int x = 0; x < 32; ++x) s[0][x] = __float_as_uint(__uint_as_float(s[0][x]) - take);
                                tc::tmem_st_32x32(tS + 32 * k, s[0]);
                            }
                            tc::tmem_st_wait();
                        }
                        if (b > b0) {  // the block before has been added: its MMA finished before this S
#pragma unroll 1
                            for (int k = 0; k < D / 32; ++k) {
                                tc::tmem_ld_32x32(tO + 32 * k, s[0]);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int x = 0; x < 32; ++x) s[0][x] = __float_as_uint(__uint_as_float(s[0][x]) * f);
                                tc::tmem_st_32x32(tO + 32 * k, s[0]);
                            }
                        }
                    }
                    const float off = fabsf(msc) >= FAR ? 0.0f : -msc;
                    const float2 sc2 = make_float2(sc, sc), off2 = make_float2(off, off);
                    uint32_t top = 0;  // bits of exp2_poly's sums
                    float2 d2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    load(0);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        tc::tmem_ld_wait();
                        if (k < 3) load(k + 1);
                        mask(k);
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            float2 e = fma2(make_float2(__uint_as_float(s[k & 1][2 * x]), __uint_as_float(s[k & 1][2 * x + 1])), sc2, off2);
                            if (x % POLY_EVERY == POLY_EVERY - 1) {
                                e = exp2_poly(e, top);
                            } else {
                                e.x = exp2_approx(e.x);
                                e.y = exp2_approx(e.y);
                            }
                            d2[x & 1] = add2(d2[x & 1], e);
                            pk[k >> 1][16 * (k & 1) + x] = pack_bf16(e.x, e.y);
                        }
                    }
                    sum = (d2[0].x + d2[0].y) + (d2[1].x + d2[1].y);
                    if (again || !__any_sync(0xffffffffu, sum > RAISE_SUM || (top ^ POLY_MAGIC) > 0xFFu || (mx == -INFINITY && seen > 0))) break;
                    again = true;
                }
                tc::tmem_st_32x32(tS, pk[0]);
                tc::tmem_st_32x32(tS + 32, pk[1]);
                den += sum;
                tc::tmem_st_wait();
                tc::fence_before_sync();
                tc::mbar_arrive(pfull(i));
            }
            // this piece's rows, before the next piece's take their place
            const bool whole = starts && ends;
            const int64_t row = row_out;
            const size_t slot_at = (size_t)(2 * c + (starts ? 1 : 0)) * C::SLOT;
            const bool piece_sees = limit > b0 * BLK;
            if (ok) {
                have = fetch();
                ok = !*aborted && tc::mbar_wait(ofull(i), no & 1, WAIT_NS);
                ok = __all_sync(0xffffffffu, ok);
                ++no;
            }
            if (!ok) {
                give_up();
                break;
            }
            tc::fence_after_sync();
            // no sum: no key in sight, or every score was -inf, which has no softmax
            const float inv = den == 0.0f ? (piece_sees ? NAN : 0.0f) : 1.0f / den;
            float4* slot = reinterpret_cast<float4*>(a.slots + slot_at) + i * TM + r;
            // whole rows go out through the tile's query memory, which no MMA reads any more
            uint32_t ov[2][32];
            tc::tmem_ld_32x32(tO, ov[0]);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                uint32_t(&o)[32] = ov[k & 1];
                tc::tmem_ld_wait();
                if (k + 1 < D / 32) tc::tmem_ld_32x32(tO + 32 * (k + 1), ov[(k + 1) & 1]);
#pragma unroll
                for (int x = 0; x < 32; x += 8) {
                    float f[8];  // back in order: column 2j is dim j, column 2j + 1 dim j + 4
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f[j] = __uint_as_float(o[x + 2 * j]);
                        f[j + 4] = __uint_as_float(o[x + 2 * j + 1]);
                    }
                    const int o8 = 4 * k + x / 8;  // octet of dims
                    if (whole) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] *= inv;
                        *cell(r, o8) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
                    } else {
                        slot[2 * o8 * ROWS] = make_float4(f[0], f[1], f[2], f[3]);
                        slot[(2 * o8 + 1) * ROWS] = make_float4(f[4], f[5], f[6], f[7]);
                    }
                }
            }
            if (whole) {
                __syncwarp();
#pragma unroll 4
                for (int x = 0; x < QN; ++x) {
                    const int from = x * RPI + lane / LPR;
                    const int64_t off = __shfl_sync(0xffffffffu, row, from);
                    if (off >= 0) *reinterpret_cast<uint4*>(a.out + off + 8 * oct) = *cell((warp & 3) * 32 + from, oct);
                }
                __syncwarp();  // the warp's own next queries go to the rows that it has just read
            } else {
                float2* st = reinterpret_cast<float2*>(a.slots + slot_at + ROWS * D) + i * TM + r;
                *st = make_float2(mx == -INFINITY ? -INFINITY : msc, den == 0.0f && piece_sees ? -0.0f : den);  // -0: as `inv` above
            }
        }
        if (tid == 0) a.joins[c] = join;
    }

    // -------------------------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && abort_sh) a.joins[c] = make_int4(0, 0, 0, GAVE_UP);
    if (warp == MMA_WARP) {
        if (abort_sh) {
            // no MMA may still be using TMEM when it is released
            if (elect_one()) tc::mma_commit(drained);
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
    bool lost = false;  // a piece saw keys, but scores of -inf only
    for (int p = 0; p < pieces; ++p) {
        const float2 st = reinterpret_cast<const float2*>(slot(p) + ROWS * D)[row];
        m = fmaxf(m, st.x);
        lost |= st.y == 0.0f && signbit(st.y);
        if (a.joins[c + p].w == GAVE_UP) return;  // a piece is missing: the item is left as it was
    }
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
    const float inv = den == 0.0f ? (lost ? NAN : 0.0f) : 1.0f / den;
    const int ri = t * ROWS + row;
    uint16_t* op = a.out + (int64_t)(j.x + ri / a.group) * a.out_stride + (j.y * a.group + ri % a.group) * D + 16 * blockIdx.y;
#pragma unroll
    for (int e = 0; e < 4; e += 2)
        *reinterpret_cast<uint4*>(op + 4 * e) =
            make_uint4(pack_bf16(v[e].x * inv, v[e].y * inv), pack_bf16(v[e].z * inv, v[e].w * inv),
                       pack_bf16(v[e + 1].x * inv, v[e + 1].y * inv), pack_bf16(v[e + 1].z * inv, v[e + 1].w * inv));
}

// The same for items of few rows, where a thread per row leaves most lanes idle and the
// pieces' latencies in line: block (c, y) takes rows 16 y .., a warp two of them, so that
// the 16 bytes of a lane and of its neighbour are a sector: lane = 2 (chunk of 4 dims) +
// row. The pieces' factors first, then their sums, eight pieces in flight. 30 pieces of
// 20 rows: 63.2 -> 56.3 us with the units' kernel; for 256 rows in 2 or 3 pieces it costs
// 2.5 us.
constexpr int FEW_ROWS = 128, JOIN_ROWS = 16;
template <int D>
__global__ void __launch_bounds__(16 * JOIN_ROWS) kv4_tile_join_few_kernel(const TileArgs a) {
    using C = Cfg<D>;
    constexpr int PER = D / 64;  // 16-byte chunks a lane, 16 apart
    __shared__ float factor[JOIN_ROWS][MAX_CTAS];
    grid_dependency_wait();
    grid_dependents_launch();
    const int4 j = a.joins[blockIdx.x];
    const int c = blockIdx.x, rows = j.z >> 20, t = j.z & 0xfffff;
    const int lane = threadIdx.x & 31, in = 2 * (threadIdx.x >> 5) + (lane & 1), row = blockIdx.y * JOIN_ROWS + in;
    if (j.w < 0 || (row & ~1) >= rows) return;
    const int pieces = j.w - c + 1, part = lane >> 1;
    auto slot = [&](int p) { return a.slots + (size_t)(2 * (c + p) + (p == 0 ? 1 : 0)) * C::SLOT; };
    auto stat = [&](int p) { return reinterpret_cast<const float2*>(slot(p) + ROWS * D)[row]; };
    float m = -INFINITY;
    int lost = 0;  // a piece saw keys, but scores of -inf only
    bool gone = false;
#pragma unroll 4
    for (int p = part; p < pieces; p += 16) {
        const float2 st = stat(p);
        m = fmaxf(m, st.x);
        lost |= st.y == 0.0f && signbit(st.y);
        gone |= a.joins[c + p].w == GAVE_UP;
    }
    if (__any_sync(0xffffffffu, gone)) return;  // a piece is missing: the item is left as it was
#pragma unroll
    for (int o = 2; o < 32; o <<= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        lost |= __shfl_xor_sync(0xffffffffu, lost, o);
    }
    float den = 0.0f;
    for (int p = part; p < pieces; p += 16) {
        const float2 st = stat(p);
        const float f = st.x == -INFINITY ? (st.y != st.y ? 1.0f : 0.0f) : exp2_approx(st.x - m);
        den += f * st.y;
        factor[in][p] = f;
    }
#pragma unroll
    for (int o = 2; o < 32; o <<= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    __syncwarp();
    float4 v[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = 0; p < pieces; ++p) {
        const float f = factor[in][p];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const float4 o = reinterpret_cast<const float4*>(slot(p))[(part + 16 * e) * ROWS + row];
            v[e].x += f * o.x, v[e].y += f * o.y, v[e].z += f * o.z, v[e].w += f * o.w;
        }
    }
    if (row >= rows) return;
    const float inv = den == 0.0f ? (lost ? NAN : 0.0f) : 1.0f / den;
    const int ri = t * ROWS + row;
    uint16_t* op = a.out + (int64_t)(j.x + ri / a.group) * a.out_stride + (j.y * a.group + ri % a.group) * D;
#pragma unroll
    for (int e = 0; e < PER; ++e)
        *reinterpret_cast<uint2*>(op + 4 * (part + 16 * e)) =
            make_uint2(pack_bf16(v[e].x * inv, v[e].y * inv), pack_bf16(v[e].z * inv, v[e].w * inv));
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
    const int64_t rows = std::min<int64_t>((int64_t)args.max_q * args.group, ROWS);
    if (rows <= FEW_ROWS)
        return launch_pdl(kv4_tile_join_few_kernel<D>, dim3((unsigned)grid, (unsigned)((rows + JOIN_ROWS - 1) / JOIN_ROWS)),
                          dim3(16 * JOIN_ROWS), 0, s, args);
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
    a.group_inv = (((uint64_t)1 << 40) + a.group - 1) / a.group;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.slots = (float*)ws;
    a.joins = (int4*)((char*)ws + (size_t)2 * MAX_CTAS * ROWS * (D + 2) * 4);
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    return D == 128 ? launch_tile<128>(a, s) : launch_tile<64>(a, s);
}

}  // namespace bl
