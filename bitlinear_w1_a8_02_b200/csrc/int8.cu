// 8-bit linear layers: int8 weights with a step per output row, int8 activations
// with a scale per token, exact int32 accumulation.
//
//   y[m, n] = [residual +] fl(fl(float(acc) wstep[n]) fl(1 / s_m))
//
// M <= 16 tokens: bound by the N K weight bytes. Warps stream 16 rows at a time
// from DRAM straight into int8 mma.sync fragments (m16n8k32, weights as A): a
// lane's 16 bytes of a row are the four words of two MMAs, and the lane's 16 bytes
// of a token's codes line up with them, so neither side is rearranged. Up to four
// tokens are quantised inside the kernel, by every block for itself.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace bl {
namespace {

constexpr int kPackThreads = 256;
constexpr float kWeightFloor = 1e-30f;

// One CTA per weight row: absmax, then codes of 4 columns per thread.
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
    for (int c = threadIdx.x; c < K / 4; c += kPackThreads) {
        load4(c, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(f[e]));
    }
    top = block_max<kPackThreads / 32>(top, scratch);
    const float step = __fdiv_rn(fmaxf(top, kWeightFloor), 127.0f);
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

__device__ __forceinline__ void store_one(const Int8Args& a, int m, int n, int acc, float wstep, float xstep) {
    const int64_t i = (int64_t)m * a.N + n;
    float f = __fmul_rn(__fmul_rn((float)acc, wstep), xstep);
    if (a.residual) f = __fadd_rn(bf16_bits_to_f32(a.residual[i]), f);
    if (a.y32)
        a.y32[i] = f;
    else
        a.y16[i] = f32_to_bf16_bits(f);
    if (a.acc) a.acc[i] = acc;
}

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kGemvWarps = 8;
constexpr int kUnroll = 5;               // 64-byte chunks of a row pair in flight per warp
constexpr int kFusedTokens = 4;          // up to here the kernel quantises x itself
constexpr int kFusedBytes = 40 * 1024;   // and keeps its codes in shared memory

struct GemvIn {
    const uint16_t* x;  // fused: activations to quantise
    int norm;
    int pitch;          // fused: bytes from one token's codes to the next
};

// The kernel's blocks are persistent and take every gridDim.x-th tile of 16 rows; the 8 warps of a block share a
// tile (64-byte chunks of K in turn), their sums meet in shared memory. The first tile's weights are under way before
// the kernel waits for the one before it: weights are constants (the header says so for packed weights).
template <int NT, bool FUSED>
__global__ void __launch_bounds__(32 * kGemvWarps, NT == 1 ? 4 : 3) gemv_int8_kernel(const Int8Args a, const GemvIn in) {
    __shared__ int part[2][kGemvWarps][NT * 4][32];
    __shared__ float xstep_sh[8 * NT];
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

    if (FUSED) {
        // as the separate quantiser does it
        for (int m = 0; m < a.M; ++m) {
            const uint4* xr = reinterpret_cast<const uint4*>(in.x + (int64_t)m * a.K);
            float top = 0.0f;
            double ss = 0.0;
            for (int c = threadIdx.x; c < a.K / 8; c += 32 * kGemvWarps) {
                const uint4 w = xr[c];
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float lo = __uint_as_float(ws[e] << 16), hi = __uint_as_float(ws[e] & 0xffff0000u);
                    top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
                    if (in.norm) ss = __fma_rn((double)lo, (double)lo, __fma_rn((double)hi, (double)hi, ss));
                }
            }
            top = block_max<kGemvWarps>(top, fscratch);
            float rms = 1.0f;
            if (in.norm) {
                ss = block_sum<kGemvWarps>(ss, dscratch);
                rms = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn((float)(ss / (double)a.K), kRmsEps)));
                top = __fmul_rn(top, rms);
            }
            const float s = __fdiv_rn(kActRange, fmaxf(top, kActEps));
            if (threadIdx.x == 0) xstep_sh[m] = __fdiv_rn(1.0f, s);
            for (int c = threadIdx.x; c < a.K / 8; c += 32 * kGemvWarps) {
                const uint4 w = xr[c];
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
                uint32_t o[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f = __uint_as_float(e & 1 ? ws[e / 2] & 0xffff0000u : ws[e / 2] << 16);
                    if (in.norm) f = __fmul_rn(f, rms);
                    o[e / 4] |= (uint32_t)(quant_code(f, s) & 255) << (8 * (e & 3));
                }
                *reinterpret_cast<uint2*>(codes + m * in.pitch + 8 * c) = make_uint2(o[0], o[1]);
            }
        }
    } else if (threadIdx.x < a.M) {
        xstep_sh[threadIdx.x] = __fdiv_rn(1.0f, a.scale[threadIdx.x]);
    }
    __syncthreads();

    const int8_t* x[NT];
    bool live[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        live[nt] = nt * 8 + r < a.M;
        const int m = min(nt * 8 + r, a.M - 1);
        x[nt] = (FUSED ? codes + m * in.pitch : a.xq + (int64_t)m * a.K) + 16 * t;
    }
    int turn = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
        // the output this thread stores after the sums have met: element e = warp of nt = 0 .. NT - 1
        const int n = tile * 16 + r + 8 * ((warp & 3) >> 1);
        const float ws = warp < 4 * NT && n < a.N ? a.wstep[n] : 0.0f;
        int d[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0;
        for (int c = warp; c < n_chunks; c += kGemvWarps * kUnroll) {
            if (c != warp || tile != blockIdx.x) load(tile, c);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int k = (c + i * kGemvWarps) * 64;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 b = k + 16 * t < a.K && live[nt] ? *reinterpret_cast<const uint4*>(x[nt] + k) : zero;
                    mma_s8(d[nt], u[i].x, v[i].x, u[i].y, v[i].y, b.x, b.y);
                    mma_s8(d[nt], u[i].z, v[i].z, u[i].w, v[i].w, b.z, b.w);
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[turn][warp][nt * 4 + e][lane] = d[nt][e];
        __syncthreads();  // the other half of `part` is free: every warp has passed the tile before
        if (warp < 4 * NT) {
            int acc = 0;
#pragma unroll
            for (int w = 0; w < kGemvWarps; ++w) acc += part[turn][w][warp][lane];
            const int m = (warp >> 2) * 8 + 2 * t + (warp & 1);
            if (n < a.N && m < a.M) store_one(a, m, n, acc, ws, xstep_sh[m]);
        }
    }
}

template <int NT, bool FUSED>
cudaError_t launch_gemv_nt(const Int8Args& a, const GemvIn& in, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static int resident[64];  // blocks the device holds at once
    if (dev >= 64 || !resident[dev]) {
        int sms = 0, per = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, gemv_int8_kernel<NT, FUSED>, 32 * kGemvWarps, FUSED ? 8192 : 0);
        if (e != cudaSuccess) return e;
        if (dev < 64) resident[dev] = sms * per;
    }
    const int tiles = (a.N + 15) / 16;
    const int grid = std::min(tiles, dev < 64 ? resident[dev] : 148);
    return launch_pdl(gemv_int8_kernel<NT, FUSED>, dim3((unsigned)grid), dim3(32 * kGemvWarps),
                      FUSED ? (size_t)in.pitch * a.M : 0, s, a, in);
}

// ---------------------------------------------------------------- M > 16: tcgen05
constexpr int BM = 128, BN = 256, BK = 128;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
constexpr int EPI_WARPS = 4;
constexpr int GEMM_THREADS = 64 + 32 * EPI_WARPS;
constexpr size_t GEMM_SMEM = 1024 + STAGES * (A_BYTES + B_BYTES) + (2 * STAGES + 4) * 8;
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;

__host__ __device__ constexpr uint32_t idesc_s8s8(int m, int n) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__global__ void __launch_bounds__(GEMM_THREADS, 1)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Int8Args a,
                     unsigned* err) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    uint8_t* sA = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sB = sA + STAGES * A_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sB + STAGES * B_BYTES);
    auto full = [&](int i) { return tc::smem_u32(bars + i); };
    auto empty = [&](int i) { return tc::smem_u32(bars + STAGES + i); };
    auto afull = [&](int i) { return tc::smem_u32(bars + 2 * STAGES + i); };
    auto aempty = [&](int i) { return tc::smem_u32(bars + 2 * STAGES + 2 + i); };
    volatile int* aborted = &abort_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_tiles = (a.N + BN - 1) / BN, m_tiles = (a.M + BM - 1) / BM;
    const int tiles = n_tiles * m_tiles, nkb = (a.K + BK - 1) / BK;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(full(i), 1), tc::mbar_init(empty(i), 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(afull(i), 1), tc::mbar_init(aempty(i), 32 * EPI_WARPS);
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
            if (*aborted)  // let the copies still in flight land before the CTA exits
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
                                          reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.acc) |
                                          reinterpret_cast<uintptr_t>(a.wstep)) % 16 == 0;
        uint32_t t = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++t) {
            const int b = t & 1;
            const bool ok = !*aborted && tc::mbar_wait(afull(b), (t >> 1) & 1, WAIT_LIMIT_NS);
            if (!__all_sync(0xffffffffu, ok)) {  // tcgen05.ld below is warp-collective
                give_up();
                break;
            }
            tc::fence_after_sync();
            const int m = (tile % m_tiles) * BM + q * 32 + lane, n0 = (tile / m_tiles) * BN;
            const bool mv = m < a.M;
            const float xstep = mv ? __fdiv_rn(1.0f, a.scale[m]) : 0.0f;
#pragma unroll 1
            for (int c = 0; c < BN / 32; ++c) {
                uint32_t v[32];
                tc::tmem_ld_32x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + b * BN + c * 32, v);
                tc::tmem_ld_wait();
                const int nb = n0 + c * 32;
                if (!mv || nb >= a.N) continue;
                const int64_t o = (int64_t)m * a.N + nb;
                if (vec && nb + 32 <= a.N) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        float f[8];
                        const float4 wa = __ldg(reinterpret_cast<const float4*>(a.wstep + nb + j));
                        const float4 wb = __ldg(reinterpret_cast<const float4*>(a.wstep + nb + j + 4));
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
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (nb + j < a.N) store_one(a, m, nb + j, (int)v[j], a.wstep[nb + j], xstep);
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
            // no MMA may still be writing TMEM when it is released
            tc::mma_commit(afull(0));
            tc::mbar_wait(afull(0), 0, WAIT_LIMIT_NS);
        }
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 2 * BN);
    }
}

}  // namespace

cudaError_t launch_pack_int8(const void* W, bool fp32, int64_t N, int64_t K, int8_t* Wq, float* wstep, cudaStream_t s) {
    if (fp32)
        pack_int8_kernel<true><<<(unsigned)N, kPackThreads, 0, s>>>(W, (int)K, Wq, wstep);
    else
        pack_int8_kernel<false><<<(unsigned)N, kPackThreads, 0, s>>>(W, (int)K, Wq, wstep);
    return cudaGetLastError();
}

cudaError_t launch_int8(const int8_t* Wq, const float* wstep, int64_t N, int64_t K, const uint16_t* x, bool rmsnorm,
                        int8_t* xq, float* scale, int64_t M, const uint16_t* residual, uint16_t* y16, float* y32, int32_t* acc,
                        cudaStream_t s) {
    Int8Args a{Wq, wstep, xq, scale, residual, y16, y32, acc, (int)M, (int)N, (int)K};
    const GemvIn in{x, rmsnorm ? 1 : 0, (int)K + 16};
    if (M <= kFusedTokens && M * in.pitch <= kFusedBytes) return launch_gemv_nt<1, true>(a, in, s);
    cudaError_t e = launch_act_quant(x, M, K, XQ_NATURAL, xq, scale, nullptr, s, rmsnorm);
    if (e != cudaSuccess) return e;
    if (M <= 8) return launch_gemv_nt<1, false>(a, in, s);
    if (M <= 16) return launch_gemv_nt<2, false>(a, in, s);
    CUtensorMap mapA, mapB;
    if (!make_map(&mapA, xq, (uint64_t)M, (uint64_t)K, BM, BK, true) ||
        !make_map(&mapB, Wq, (uint64_t)N, (uint64_t)K, BN, BK, true))
        return cudaErrorInvalidValue;
    unsigned* err = nullptr;
    e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gemm_int8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GEMM_SMEM);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((N + BN - 1) / BN) * ((M + BM - 1) / BM);
    return launch_pdl(gemm_int8_kernel, dim3((unsigned)std::min<int64_t>(tiles, sms)), dim3(GEMM_THREADS), GEMM_SMEM, s, mapA,
                      mapB, a, err);
}

}  // namespace bl
