// 8-bit linear layers: int8 weights with a step per output row, int8 activations
// with a scale per token, exact int32 accumulation.
//
//   y[m, n] = [residual +] fl(fl(float(acc) wstep[n]) fl(1 / s_m))
//
// One token: bound by the N K weight bytes. Warps stream 16 rows at a time from
// DRAM straight into int8 mma.sync fragments (m16n8k32, weights as A): a lane's 16
// bytes of a row are the four words of two MMAs, and the lane's 16 bytes of the
// token's codes line up with them, so neither side is rearranged. The token is
// quantised inside the kernel, by every block for itself: one launch, 4.1 us
// against 5.5 with a quantiser before the kernel for few tokens (2560 x 2560).
// 28672 x 8192 takes 43.6 us in a replayed graph, 5.4 TB/s of weights, 49 with
// cold caches.
//
// Packing: a block a row, read twice (the second time from L2). Bound by the
// codes' divisions: 128256 x 2560 410 us from bf16, 418 from fp32, 2.4 and 3.9
// TB/s of weights and codes.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace bl {
namespace {

constexpr int kPackThreads = 256;
constexpr float kWeightFloor = 1e-30f;

// One CTA per weight row: absmax, then codes of 4 columns per thread. A NaN, which a maximum passes over, becomes the
// row's step; the codes are zero then, as with an infinite step.
template <bool FP32>
__global__ void __launch_bounds__(kPackThreads) pack_int8_kernel(const void* W, int K, int8_t* Wq, float* wstep) {
    __shared__ float scratch[kPackThreads / 32];
    const int64_t n = blockIdx.x;
    auto load4 = [&](int c, float (&f)[4]) {
        if (FP32) {
            const float4 v = reinterpret_cast<const float4*>(static_cast<const float*>(W) + n * K)[c];
            f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
        } else {
            const uint2 v = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(W) + n * K)[c];
            f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
            f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
        }
    };
    float top = 0.0f, f[4];
    bool nan = false;
    for (int c = threadIdx.x; c < K / 4; c += kPackThreads) {
        load4(c, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            top = fmaxf(top, fabsf(f[e]));
            nan |= f[e] != f[e];
        }
    }
    top = block_max<kPackThreads / 32>(top, scratch);
    const float step = __syncthreads_or(nan) ? NAN : __fdiv_rn(fmaxf(top, kWeightFloor), 127.0f);
    for (int c = threadIdx.x; c < K / 4; c += kPackThreads) {
        load4(c, f);
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int q = (int)rintf(__fdiv_rn(f[e], step));
            w |= (uint32_t)(min(max(q, -127), 127) & 255) << (8 * e);
        }
        reinterpret_cast<uint32_t*>(Wq + n * K)[c] = w;
    }
    if (threadIdx.x == 0) wstep[n] = step;
}

struct Int8Args {
    const int8_t* Wq;
    const float* wstep;
    const int8_t* xq;
    const float* scale;
    const uint16_t* residual;
    uint16_t* y16;
    float* y32;
    int32_t* acc;
    int M, N, K;
};

// Output i of the sum acc, whose scaled value is f.
__device__ __forceinline__ void put_one(const Int8Args& a, int64_t i, int acc, float f) {
    if (a.residual) f = __fadd_rn(bf16_bits_to_f32(a.residual[i]), f);
    if (a.y32)
        a.y32[i] = f;
    else
        a.y16[i] = f32_to_bf16_bits(f);
    if (a.acc) a.acc[i] = acc;
}

__device__ __forceinline__ void store_one(const Int8Args& a, int m, int n, int acc, float wstep, float xstep) {
    put_one(a, (int64_t)m * a.N + n, acc, __fmul_rn(__fmul_rn((float)acc, wstep), xstep));
}

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kGemvWarps = 8;
constexpr int kUnroll = 5;              // 64-byte chunks of a row pair in flight per warp
constexpr int kGemvMaxK = 32 * 1024;    // its codes stay in shared memory, 48 KiB with the static part
// Many short rows go to the kernel for few tokens instead, whose tiles of 128 rows meet less often (one token, here
// against there): 4096 x 256 2.7 and 4.1 us, 16384 x 768 6.5 and 7.1, 32768 x 2048 14.8 and 15.7; 16384 x 256 4.4 and
// 4.2, 32768 x 1024 10.8 and 10.0, 80000 x 768 18.7 and 14.9, 128256 x 2560 53.3 and 52.0.
constexpr int64_t kGemvRows = 8192, kGemvRatio = 24;

// The kernel's blocks are persistent and take every gridDim.x-th tile of 16 rows; the 8 warps of a block share a
// tile (64-byte chunks of K in turn), their sums meet in shared memory. The first tile's weights are under way before
// the kernel waits for the one before it: weights are constants (the header says so for packed weights).
__global__ void __launch_bounds__(32 * kGemvWarps, 4) gemv_int8_kernel(const Int8Args a, const uint16_t* x, int norm) {
    __shared__ int part[2][kGemvWarps][16];
    __shared__ float fscratch[kGemvWarps];
    __shared__ double dscratch[kGemvWarps];
    extern __shared__ __align__(16) int8_t codes[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, t = lane & 3;
    const int tiles = (a.N + 15) / 16;
    const int n_chunks = (a.K + 63) / 64;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 u[kUnroll], v[kUnroll];
    // chunks c, c + 8, ... of tile `tile`; rows past the end read row N - 1, and their sums are not stored
    auto load = [&](int tile, int c) {
        const int8_t* w0 = a.Wq + (int64_t)min(tile * 16 + r, a.N - 1) * a.K + 16 * t;
        const int8_t* w1 = a.Wq + (int64_t)min(tile * 16 + r + 8, a.N - 1) * a.K + 16 * t;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int k = (c + i * kGemvWarps) * 64;
            const bool in_k = k + 16 * t < a.K;  // K is a multiple of 16
            u[i] = in_k ? ld_stream16(w0 + k) : zero;
            v[i] = in_k ? ld_stream16(w1 + k) : zero;
        }
    };
    load(blockIdx.x, warp);
    grid_dependency_wait();
    grid_dependents_launch();

    // the codes, as the separate quantiser makes them
    const uint4* xr = reinterpret_cast<const uint4*>(x);
    float top = 0.0f;
    double ss = 0.0;
    for (int c = threadIdx.x; c < a.K / 8; c += 32 * kGemvWarps) {
        const uint4 w = xr[c];
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float lo = __uint_as_float(ws[e] << 16), hi = __uint_as_float(ws[e] & 0xffff0000u);
            top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
            if (norm) ss = __fma_rn((double)lo, (double)lo, __fma_rn((double)hi, (double)hi, ss));
        }
    }
    top = block_max<kGemvWarps>(top, fscratch);
    float rms = 1.0f;
    if (norm) {
        ss = block_sum<kGemvWarps>(ss, dscratch);
        rms = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn((float)(ss / (double)a.K), kRmsEps)));
        top = __fmul_rn(top, rms);
    }
    const float s = __fdiv_rn(kActRange, fmaxf(top, kActEps)), xstep = __fdiv_rn(1.0f, s);
    for (int c = threadIdx.x; c < a.K / 8; c += 32 * kGemvWarps) {
        const uint4 w = xr[c];
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float f = __uint_as_float(e & 1 ? ws[e / 2] & 0xffff0000u : ws[e / 2] << 16);
            if (norm) f = __fmul_rn(f, rms);
            o[e / 4] |= (uint32_t)(quant_code(f, s) & 255) << (8 * (e & 3));
        }
        *reinterpret_cast<uint2*>(codes + 8 * c) = make_uint2(o[0], o[1]);
    }
    __syncthreads();

    int turn = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
        const int n = tile * 16 + (int)threadIdx.x;  // the row this thread finishes, if it is one of the first 16
        const bool last = threadIdx.x < 16 && n < a.N;
        const float ws = last ? a.wstep[n] : 0.0f;
        int d[4] = {0, 0, 0, 0};  // the token is column 0: d[0] and d[2] of lanes with t = 0
        for (int c = warp; c < n_chunks; c += kGemvWarps * kUnroll) {
            if (c != warp || tile != blockIdx.x) load(tile, c);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int k = (c + i * kGemvWarps) * 64 + 16 * t;
                const uint4 b = k < a.K && r == 0 ? *reinterpret_cast<const uint4*>(codes + k) : zero;
                mma_s8(d, u[i].x, v[i].x, u[i].y, v[i].y, b.x, b.y);
                mma_s8(d, u[i].z, v[i].z, u[i].w, v[i].w, b.z, b.w);
            }
        }
        if (t == 0) part[turn][warp][r] = d[0], part[turn][warp][r + 8] = d[2];
        __syncthreads();  // the other half of `part` is free: every warp has passed the tile before
        if (last) {
            int acc = 0;
#pragma unroll
            for (int w = 0; w < kGemvWarps; ++w) acc += part[turn][w][threadIdx.x];
            store_one(a, 0, n, acc, ws, xstep);
        }
    }
}

cudaError_t launch_gemv(const Int8Args& a, const uint16_t* x, bool norm, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static int resident[64];  // blocks the device holds at once
    if (dev >= 64 || !resident[dev]) {
        int sms = 0, per = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, gemv_int8_kernel, 32 * kGemvWarps, 8192);
        if (e != cudaSuccess) return e;
        if (dev < 64) resident[dev] = sms * per;
    }
    const int tiles = (a.N + 15) / 16;
    const int grid = std::min(tiles, dev < 64 ? resident[dev] : 148);
    return launch_pdl(gemv_int8_kernel, dim3((unsigned)grid), dim3(32 * kGemvWarps), (size_t)a.K, s, a, x, norm ? 1 : 0);
}

// ---------------------------------------------------------------- M > 128: tcgen05
//
// M > 128: TMA brings 128 bytes of K of 128 tokens and BN weight rows per stage, one thread issues tcgen05.mma kind::i8
// into one of two int32 accumulators in TMEM, eight warps read the other one out. Persistent blocks take whole tiles;
// weight tiles are shared by consecutive tiles. Bound by the tensor work: 2048 tokens 8192 -> 28672 341 us, 2.8 POP/s,
// the tensor pipe 77% busy; where there is a tile or less to an SM, by the latency of its loads: 2560 -> 2560 with 300
// tokens 11.2 us.
constexpr int BM = 128, BK = 128;
constexpr int A_BYTES = BM * BK;
constexpr int EPI_WARPS = 8;  // two to a quarter of TMEM's lanes, 32 columns in turn
constexpr int GEMM_THREADS = 64 + 32 * EPI_WARPS;
template <int BN>
struct Gemm {
    static constexpr int B_BYTES = BN * BK;
    static constexpr int STAGES = BN == 256 ? 4 : 6;
    static constexpr int BARS = 2 * STAGES + 5;
    static constexpr size_t SMEM = 1024 + STAGES * (A_BYTES + B_BYTES) + BARS * 8;
    static_assert(SMEM + EPI_WARPS * 4 * (16 * 33 + BN) + 16 <= 227 * 1024, "shared memory of a block");
};
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;

__host__ __device__ constexpr uint32_t idesc_s8s8(int m, int n) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <int BN>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Int8Args a,
                     unsigned* err) {
    constexpr int STAGES = Gemm<BN>::STAGES, B_BYTES = Gemm<BN>::B_BYTES;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    __shared__ int turn_sh[EPI_WARPS][16][33];
    __shared__ __align__(16) float ws_sh[EPI_WARPS][BN];  // a warp's copy of the tile's weight steps
    uint8_t* sA = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sB = sA + STAGES * A_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sB + STAGES * B_BYTES);
    auto full = [&](int i) { return tc::smem_u32(bars + i); };
    auto empty = [&](int i) { return tc::smem_u32(bars + STAGES + i); };
    auto afull = [&](int i) { return tc::smem_u32(bars + 2 * STAGES + i); };
    auto aempty = [&](int i) { return tc::smem_u32(bars + 2 * STAGES + 2 + i); };
    const uint32_t drained = tc::smem_u32(bars + 2 * STAGES + 4);  // teardown after an abort
    volatile int* aborted = &abort_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_tiles = (a.N + BN - 1) / BN, m_tiles = (a.M + BM - 1) / BM;
    const int tiles = n_tiles * m_tiles, nkb = (a.K + BK - 1) / BK;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(full(i), 1), tc::mbar_init(empty(i), 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(afull(i), 1), tc::mbar_init(aempty(i), 32 * EPI_WARPS);
        tc::mbar_init(drained, 1);
        abort_sh = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tc::smem_u32(&tmem_base_sh), 2 * BN);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base_sh;
    grid_dependency_wait();
    grid_dependents_launch();
    auto give_up = [&]() {
        atomicOr(err, 1u);
        *aborted = 1;
    };
    if (warp == 0) {
        if (lane == 0) {
            asm volatile("fence.proxy.async.global;" ::: "memory");  // codes written by the kernel before
            uint32_t g = 0;
            for (int tile = blockIdx.x; tile < tiles && !*aborted; tile += gridDim.x) {
                const int m0 = (tile % m_tiles) * BM, n0 = (tile / m_tiles) * BN;
                for (int kb = 0; kb < nkb; ++kb, ++g) {
                    const int s = g % STAGES;
                    if (g >= STAGES && !tc::mbar_wait(empty(s), (g / STAGES - 1) & 1, WAIT_LIMIT_NS)) {
                        give_up();
                        break;
                    }
                    tc::mbar_arrive_expect_tx(full(s), A_BYTES + B_BYTES);
                    tc::tma_load_2d(tc::smem_u32(sA + s * A_BYTES), &tmA, kb * BK, m0, full(s));
                    tc::tma_load_2d(tc::smem_u32(sB + s * B_BYTES), &tmB, kb * BK, n0, full(s));
                }
            }
            // let the copies still in flight land before the CTA exits: the MMA thread waits for them too, unless it gives up
            for (uint32_t h = g > STAGES ? g - STAGES : 0; h < g; ++h)
                tc::mbar_wait(full(h % STAGES), (h / STAGES) & 1, WAIT_LIMIT_NS);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_s8s8(BM, BN);
            uint32_t g = 0, t = 0;
            for (int tile = blockIdx.x; tile < tiles && !*aborted; tile += gridDim.x, ++t) {
                const int b = t & 1;
                bool ok = t < 2 || tc::mbar_wait(aempty(b), ((t >> 1) - 1) & 1, WAIT_LIMIT_NS);
                tc::fence_after_sync();
                for (int kb = 0; ok && kb < nkb; ++kb, ++g) {
                    const int s = g % STAGES;
                    ok = tc::mbar_wait(full(s), (g / STAGES) & 1, WAIT_LIMIT_NS);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint64_t ad = tc::desc_kmajor_sw128(tc::smem_u32(sA + s * A_BYTES));
                    const uint64_t bd = tc::desc_kmajor_sw128(tc::smem_u32(sB + s * B_BYTES));
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        tc::mma_i8(tmem + b * BN, ad + 2 * kk, bd + 2 * kk, idesc, kb != 0 || kk != 0);
                    tc::mma_commit(empty(s));
                }
                if (!ok) {
                    give_up();
                    break;
                }
                tc::mma_commit(afull(b));
            }
        }
    } else {
        const int q = warp & 3;  // the TMEM lane quarter this warp may read
        const bool vec = a.N % 8 == 0 && (reinterpret_cast<uintptr_t>(a.y16) | reinterpret_cast<uintptr_t>(a.y32) |
                                          reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.acc)) % 16 == 0;
        uint32_t t = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++t) {
            const int b = t & 1;
            const int m = (tile % m_tiles) * BM + q * 32 + lane, n0 = (tile / m_tiles) * BN;
            const bool mv = m < a.M;
            const float xstep = mv ? __fdiv_rn(1.0f, a.scale[m]) : 0.0f;
            __syncwarp();
            for (int c = lane; c < BN; c += 32) ws_sh[warp - 2][c] = n0 + c < a.N ? a.wstep[n0 + c] : 0.0f;
            __syncwarp();
            const bool ok = !*aborted && tc::mbar_wait(afull(b), (t >> 1) & 1, WAIT_LIMIT_NS);
            if (!__all_sync(0xffffffffu, ok)) {  // tcgen05.ld below is warp-collective
                give_up();
                break;
            }
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = (warp - 2) / 4; c < BN / 32; c += EPI_WARPS / 4) {
                uint32_t v[32];
                tc::tmem_ld_32x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + b * BN + c * 32, v);
                tc::tmem_ld_wait();
                const int nb = n0 + c * 32;
                if (nb >= a.N) break;
                if (!vec || nb + 32 > a.N) {
                    // rows without 16-byte alignment: through shared memory, so that a lane has a column and a warp
                    // stores 32 neighbouring values of a row
                    int(&turn)[16][33] = turn_sh[warp - 2];
                    const int n = nb + lane, m0 = m - lane, rows = min(32, a.M - m0);
                    const float ws = ws_sh[warp - 2][c * 32 + lane];
                    const int64_t o = (int64_t)m0 * a.N + n;
                    const bool plain = a.y16 && !a.residual && !a.acc;
                    for (int r0 = 0; r0 < rows; r0 += 8) {
                        if (r0 % 16 == 0) {
                            __syncwarp();
                            if (lane / 16 == r0 / 16) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) turn[lane & 15][j] = (int)v[j];
                            }
                            __syncwarp();
                        }
                        int acc[8];
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            acc[e] = turn[(r0 & 15) + e][lane];
                            f[e] = __fmul_rn(__fmul_rn((float)acc[e], ws), __shfl_sync(0xffffffffu, xstep, r0 + e));
                        }
                        if (n >= a.N) continue;
                        if (plain) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (r0 + e < rows) a.y16[o + (int64_t)(r0 + e) * a.N] = f32_to_bf16_bits(f[e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (r0 + e < rows) put_one(a, o + (int64_t)(r0 + e) * a.N, acc[e], f[e]);
                        }
                    }
                    continue;
                }
                if (!mv) continue;
                const int64_t o = (int64_t)m * a.N + nb;
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    float f[8];
                    const float4 wa = *reinterpret_cast<const float4*>(&ws_sh[warp - 2][c * 32 + j]);
                    const float4 wb = *reinterpret_cast<const float4*>(&ws_sh[warp - 2][c * 32 + j + 4]);
                    const float ws[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(__fmul_rn((float)(int)v[j + e], ws[e]), xstep);
                    if (a.residual) {
                        const uint4 rr = *reinterpret_cast<const uint4*>(a.residual + o + j);
                        const uint32_t rw[4] = {rr.x, rr.y, rr.z, rr.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f[2 * e] = __fadd_rn(bf16_bits_to_f32(rw[e] & 0xffffu), f[2 * e]);
                            f[2 * e + 1] = __fadd_rn(bf16_bits_to_f32(rw[e] >> 16), f[2 * e + 1]);
                        }
                    }
                    if (a.y32) {
                        *reinterpret_cast<float4*>(a.y32 + o + j) = make_float4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<float4*>(a.y32 + o + j + 4) = make_float4(f[4], f[5], f[6], f[7]);
                    } else {
                        uint32_t pk[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            pk[e] = f32_to_bf16_bits(f[2 * e]) | (uint32_t)f32_to_bf16_bits(f[2 * e + 1]) << 16;
                        *reinterpret_cast<uint4*>(a.y16 + o + j) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                    if (a.acc) {
                        *reinterpret_cast<int4*>(a.acc + o + j) = make_int4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                        *reinterpret_cast<int4*>(a.acc + o + j + 4) = make_int4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
                    }
                }
            }
            tc::fence_before_sync();
            tc::mbar_arrive(aempty(b));
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        if (lane == 0 && abort_sh) {
            // no MMA may still be writing TMEM when it is released (a barrier of its own: the others have phases behind them)
            tc::mma_commit(drained);
            tc::mbar_wait(drained, 0, WAIT_LIMIT_NS);
        }
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 2 * BN);
    }
}

// ---------------------------------------------------------------- up to 128 tokens: tcgen05, weights as A
//
// Bound by the weights' bytes, so every SM has to stream its share: a block takes 128 weight rows (the MMA's M) and the
// tokens are its N, and where there are fewer tiles of 128 rows than SMs, the blocks of a cluster take a K range of one
// tile each. Their int32 sums meet through distributed shared memory: each block finishes its share of the rows.
// Weight loads start before the kernel waits for the one before it. 16 tokens 8192 -> 28672: 45 us with cold caches, 5.2
// TB/s; 2560 -> 6912 7 us with the quantiser, most of it the two kernels' latencies.
constexpr int FEW_MAX = 128;
constexpr int FEW_EPI = 128, FEW_THREADS = 64 + FEW_EPI;
constexpr int FEW_SMEM = 104 * 1024, FEW_SMEM_TALL = 55 * 1024;  // two and four blocks per SM
constexpr int FEW_STAGES_MAX = 6;

struct FewArgs {
    int stages, cols, log_split;  // ring stages, tokens rounded up to 16, log2 of the blocks per tile
};

__device__ __forceinline__ int4 ld_cluster(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A block's share of its tile's rows, of 2^LS blocks' sums [token][128 rows] in shared memory: a thread keeps four
// neighbouring rows.
template <int LS>
__device__ __forceinline__ void finish_rows(const Int8Args& a, const int* sums, const float* xstep, int n0, int rank, int et) {
    constexpr int ROWS = BM >> LS, QUADS = ROWS / 4;
    const int row = rank * ROWS + et % QUADS * 4, n = n0 + row;
    if (n >= a.N) return;
    const bool vec = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y16) | reinterpret_cast<uintptr_t>(a.y32) |
                                      reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.acc)) % 16 == 0;
    float ws[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) ws[e] = n + e < a.N ? a.wstep[n + e] : 0.0f;
    uint32_t at[1 << LS];
#pragma unroll
    for (int p = 0; p < 1 << LS; ++p) at[p] = LS ? tc::map_to_rank(tc::smem_u32(sums + row), p) : 0;
#pragma unroll 1
    for (int m = et / QUADS; m < a.M; m += FEW_EPI / QUADS) {
        int v[4];
        if constexpr (LS == 0) {
            const int4 x = *reinterpret_cast<const int4*>(sums + m * BM + row);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            int4 x[1 << LS];
#pragma unroll
            for (int p = 0; p < 1 << LS; ++p) x[p] = ld_cluster(at[p] + m * BM * 4);
            v[0] = v[1] = v[2] = v[3] = 0;
#pragma unroll
            for (int p = 0; p < 1 << LS; ++p) v[0] += x[p].x, v[1] += x[p].y, v[2] += x[p].z, v[3] += x[p].w;
        }
        if (!vec) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.N) store_one(a, m, n + e, v[e], ws[e], xstep[m]);
            continue;
        }
        const int64_t o = (int64_t)m * a.N + n;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __fmul_rn(__fmul_rn((float)v[e], ws[e]), xstep[m]);
        if (a.residual) {
            const uint2 r = *reinterpret_cast<const uint2*>(a.residual + o);
            y[0] = __fadd_rn(bf16_bits_to_f32(r.x & 0xffffu), y[0]);
            y[1] = __fadd_rn(bf16_bits_to_f32(r.x >> 16), y[1]);
            y[2] = __fadd_rn(bf16_bits_to_f32(r.y & 0xffffu), y[2]);
            y[3] = __fadd_rn(bf16_bits_to_f32(r.y >> 16), y[3]);
        }
        if (a.y32)
            *reinterpret_cast<float4*>(a.y32 + o) = make_float4(y[0], y[1], y[2], y[3]);
        else
            *reinterpret_cast<uint2*>(a.y16 + o) = make_uint2(f32_to_bf16_bits(y[0]) | (uint32_t)f32_to_bf16_bits(y[1]) << 16,
                                                              f32_to_bf16_bits(y[2]) | (uint32_t)f32_to_bf16_bits(y[3]) << 16);
        if (a.acc) *reinterpret_cast<int4*>(a.acc + o) = make_int4(v[0], v[1], v[2], v[3]);
    }
}

__global__ void __launch_bounds__(FEW_THREADS)
    few_int8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Int8Args a,
                    const FewArgs f, unsigned* err) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * FEW_STAGES_MAX + 1];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    __shared__ float xstep_sh[FEW_MAX];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int x_bytes = f.cols * BK, stage_bytes = A_BYTES + x_bytes;
    auto full = [&](int i) { return tc::smem_u32(bars + i); };
    auto empty = [&](int i) { return tc::smem_u32(bars + FEW_STAGES_MAX + i); };
    const uint32_t done = tc::smem_u32(bars + 2 * FEW_STAGES_MAX);
    volatile int* aborted = &abort_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x & ((1 << f.log_split) - 1), n0 = (int)(blockIdx.x >> f.log_split) * BM;
    const int nkb = (a.K + BK - 1) / BK;
    const int kb0 = nkb * rank >> f.log_split, kb1 = nkb * (rank + 1) >> f.log_split;
    if (threadIdx.x == 0) {
        for (int i = 0; i < f.stages; ++i) tc::mbar_init(full(i), 1), tc::mbar_init(empty(i), 1);
        tc::mbar_init(done, 1);
        abort_sh = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tc::smem_u32(&tmem_base_sh), 128);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base_sh;
    auto give_up = [&]() {
        atomicOr(err, 1u);
        *aborted = 1;
    };
    if (warp == 0) {
        if (lane == 0) {
            auto weights = [&](int kb, int s) {
                tc::mbar_arrive_expect_tx(full(s), stage_bytes);
                tc::tma_load_2d(tc::smem_u32(ring + s * stage_bytes), &tmW, kb * BK, n0, full(s));
            };
            auto tokens = [&](int kb, int s) {
                tc::tma_load_2d(tc::smem_u32(ring + s * stage_bytes + A_BYTES), &tmX, kb * BK, 0, full(s));
            };
            const int ahead = min(f.stages, kb1 - kb0);
            for (int i = 0; i < ahead; ++i) weights(kb0 + i, i);
            grid_dependency_wait();
            grid_dependents_launch();
            asm volatile("fence.proxy.async.global;" ::: "memory");  // codes written by the kernel before
            for (int i = 0; i < ahead; ++i) tokens(kb0 + i, i);
            int g = ahead;
            for (int kb = kb0 + ahead; kb < kb1 && !*aborted; ++kb, ++g) {
                const int s = g % f.stages;
                if (!tc::mbar_wait(empty(s), (g / f.stages - 1) & 1, WAIT_LIMIT_NS)) {
                    give_up();
                    break;
                }
                weights(kb, s);
                tokens(kb, s);
            }
            // let the copies still in flight land before the block exits, as above
            for (int h = max(0, g - f.stages); h < g; ++h) tc::mbar_wait(full(h % f.stages), (h / f.stages) & 1, WAIT_LIMIT_NS);
        }
    } else if (warp == 1) {
        grid_dependency_wait();
        if (lane == 0) {
            const uint32_t idesc = idesc_s8s8(BM, 16) - (2u << 17) + (static_cast<uint32_t>(f.cols >> 3) << 17);
            bool ok = true;
            for (int g = 0; g < kb1 - kb0; ++g) {
                const int s = g % f.stages;
                ok = !*aborted && tc::mbar_wait(full(s), (g / f.stages) & 1, WAIT_LIMIT_NS);
                if (!ok) break;
                tc::fence_after_sync();
                const uint64_t wd = tc::desc_kmajor_sw128(tc::smem_u32(ring + s * stage_bytes));
                const uint64_t xd = tc::desc_kmajor_sw128(tc::smem_u32(ring + s * stage_bytes + A_BYTES));
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk) tc::mma_i8(tmem, wd + 2 * kk, xd + 2 * kk, idesc, g != 0 || kk != 0);
                tc::mma_commit(empty(s));
            }
            if (!ok) give_up();
            tc::mma_commit(done);
        }
        __syncwarp();
    } else {
        grid_dependency_wait();
        const int m = threadIdx.x - 64;
        if (m < a.M) xstep_sh[m] = __fdiv_rn(1.0f, a.scale[m]);
    }
    // the sums -> shared memory [token][weight row] (the ring is no longer in use)
    const bool ok = tc::mbar_wait(done, 0, 2 * WAIT_LIMIT_NS) && !*aborted;
    if (!__all_sync(0xffffffffu, ok)) give_up();
    tc::fence_after_sync();
    int* sums = reinterpret_cast<int*>(ring);
    const bool have = __all_sync(0xffffffffu, ok && !*aborted);
    if (warp >= 2 && !have) {
        // no block of the cluster can finish its rows: they all learn of it before they meet
        if (lane < 1 << f.log_split) st_cluster(tc::map_to_rank(tc::smem_u32(&abort_sh), lane), 1);
    }
    if (warp >= 2 && have) {
        const int q = warp & 3;  // the TMEM lane quarter this warp may read
        for (int c = 0; c < f.cols; c += 16) {
            uint32_t v[16];
            tc::tmem_ld_32x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
            tc::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) sums[(c + j) * BM + q * 32 + lane] = (int)v[j];
        }
    }
    tc::fence_before_sync();
    if (f.log_split)
        tc::cluster_sync();
    else
        __syncthreads();
    if (warp >= 2 && !*aborted) {
        const int et = threadIdx.x - 64;
        switch (f.log_split) {
            case 0: finish_rows<0>(a, sums, xstep_sh, n0, rank, et); break;
            case 1: finish_rows<1>(a, sums, xstep_sh, n0, rank, et); break;
            case 2: finish_rows<2>(a, sums, xstep_sh, n0, rank, et); break;
            default: finish_rows<3>(a, sums, xstep_sh, n0, rank, et);
        }
    }
    if (f.log_split)
        tc::cluster_sync();  // the others have read this block's sums
    else
        __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc(tmem, 128);
}

cudaError_t launch_few(const Int8Args& a, int sms, int dev, cudaStream_t s) {
    FewArgs f;
    f.cols = (a.M + 15) / 16 * 16;
    const int stage = A_BYTES + f.cols * BK;
    const int tiles = (a.N + BM - 1) / BM, nkb = (a.K + BK - 1) / BK;
    // Up to 8 blocks per tile with at least two k-blocks each, one block per SM. Two blocks per SM save half a block's
    // loads and make the meeting of the sums dearer, the more tokens the more: with 4 k-blocks left each (K = 4096)
    // 8.4 against 8.7 us for 16 tokens, but 13.6 against 11.7 for 128; with 6.75 (K = 6912) 14.6 against 15.2 for 128.
    f.log_split = 0;
    for (; f.log_split < 3; ++f.log_split) {
        const int blocks = tiles << (f.log_split + 1), least = blocks <= sms ? 2 : std::min(2 + f.cols / 16, 6);
        if (blocks > 2 * sms || nkb < least << (f.log_split + 1)) break;
    }
    // Deep rings where every block is resident; else (up to 64 tokens: many_rows takes the others) twice the blocks per SM
    // with two stages or three, so that some load while others start or finish: 2560 -> 128256 with 2 tokens 57.3 -> 52.0 us,
    // with 64 69.0 -> 61.8.
    f.stages = std::min(FEW_STAGES_MAX, ((tiles <= 2 * sms ? FEW_SMEM : FEW_SMEM_TALL) - 1024) / stage);
    CUtensorMap mapW, mapX;
    if (!make_map(&mapW, a.Wq, (uint64_t)a.N, (uint64_t)a.K, BM, BK, true) ||
        !make_map(&mapX, a.xq, (uint64_t)a.M, (uint64_t)a.K, (uint32_t)f.cols, BK, true))
        return cudaErrorInvalidValue;
    unsigned* err = nullptr;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    static bool attr_set[64];
    if (dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(few_int8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles << f.log_split));
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = (size_t)1024 + f.stages * stage;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << f.log_split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_int8_kernel, mapW, mapX, a, f, err);
}

template <int BN>
cudaError_t launch_gemm_bn(const Int8Args& a, int sms, int dev, cudaStream_t s) {
    CUtensorMap mapA, mapB;
    if (!make_map(&mapA, a.xq, (uint64_t)a.M, (uint64_t)a.K, BM, BK, true) ||
        !make_map(&mapB, a.Wq, (uint64_t)a.N, (uint64_t)a.K, BN, BK, true))
        return cudaErrorInvalidValue;
    unsigned* err = nullptr;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    static bool attr_set[64];
    if (dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(gemm_int8_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Gemm<BN>::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    const int64_t tiles = (int64_t)((a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM);
    return launch_pdl(gemm_int8_kernel<BN>, dim3((unsigned)std::min<int64_t>(tiles, sms)), dim3(GEMM_THREADS), Gemm<BN>::SMEM, s,
                      mapA, mapB, a, err);
}

}  // namespace

cudaError_t launch_pack_int8(const void* W, bool fp32, int64_t N, int64_t K, int8_t* Wq, float* wstep, cudaStream_t s) {
    if (fp32)
        pack_int8_kernel<true><<<(unsigned)N, kPackThreads, 0, s>>>(W, (int)K, Wq, wstep);
    else
        pack_int8_kernel<false><<<(unsigned)N, kPackThreads, 0, s>>>(W, (int)K, Wq, wstep);
    return cudaGetLastError();
}

namespace {
// 65 to 128 tokens: tiles of tokens (below) rather than of weights where these fill the SMs without a K split, or nearly
// so with short rows. In us, tiles of weights against of tokens, 96 tokens: 2560 -> 6912 12.4 and 10.8, 2560 -> 13824
// 15.0 and 12.4, 2560 -> 128256 74.9 and 63.5, 1024 -> 9000 10.1 and 8.3; 6912 -> 2560 12.9 and 19.1, 8192 -> 8192 19.9
// and 24.1. With 33 tokens: 2560 -> 6912 9.6 and 12.6, 2560 -> 128256 56.9 and 70.5.
bool many_rows(int64_t M, int64_t N, int64_t K, int sms) {
    const int64_t tiles = (N + BM - 1) / BM;
    return M > 64 && (tiles > sms || (3 * tiles >= sms && K <= 4096));
}

// 256 weight rows a tile unless narrower ones finish sooner: waves times the relative time of a tile. In us for 64, 128
// and 256 rows: 2560 x 2560 with 300 tokens 11.2, 12.1, 14.6; 6912 x 2560 with 256 tokens 16.3, 12.9, 15.7; 8192 x
// 8192 with 800 tokens 126, 78, 57. Of 63 shapes measured the pick was 9% off at worst (6919 x 2560 with 800 tokens).
int int8_tile_width(int64_t M, int64_t N, int sms) {
    const int64_t mt = (M + BM - 1) / BM;
    const int width[3] = {256, 128, 64};
    const double cost[3] = {1.0, 0.68, 0.59};
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < 3; ++i) {
        const double t = (double)((mt * ((N + width[i] - 1) / width[i]) + sms - 1) / sms) * cost[i];
        if (i == 0 || t < least - 1e-9) best = i, least = t;
    }
    return width[best];
}
}  // namespace

cudaError_t launch_int8(const int8_t* Wq, const float* wstep, int64_t N, int64_t K, const uint16_t* x, bool rmsnorm,
                        int8_t* xq, float* scale, int64_t M, const uint16_t* residual, uint16_t* y16, float* y32, int32_t* acc,
                        cudaStream_t s) {
    Int8Args a{Wq, wstep, xq, scale, residual, y16, y32, acc, (int)M, (int)N, (int)K};
    // the one-token kernel's blocks read x while others already write, so an output in x's place takes the other kernels,
    // which have x quantised before they start
    const bool in_place = overlap(x, 2 * K, y16, 2 * N) || overlap(x, 2 * K, y32, 4 * N) || overlap(x, 2 * K, acc, 4 * N);
    if (M == 1 && K <= kGemvMaxK && (N <= kGemvRows || N <= kGemvRatio * K) && !in_place) return launch_gemv(a, x, rmsnorm, s);
    cudaError_t e = launch_act_quant(x, M, K, XQ_NATURAL, xq, scale, nullptr, s, rmsnorm);
    if (e != cudaSuccess) return e;
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static int num_sms[64];
    int sms = dev < 64 ? num_sms[dev] : 0;
    if (!sms) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (dev < 64) num_sms[dev] = sms;
    }
    if (M <= FEW_MAX && !many_rows(M, N, K, sms)) return launch_few(a, sms, dev, s);
    switch (int8_tile_width(M, N, sms)) {
        case 64: return launch_gemm_bn<64>(a, sms, dev, s);
        case 128: return launch_gemm_bn<128>(a, sms, dev, s);
        default: return launch_gemm_bn<256>(a, sms, dev, s);
    }
}

}  // namespace bl
