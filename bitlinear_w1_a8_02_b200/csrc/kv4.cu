// Append to and read from the 4-bit paged cache.
//
// Append: one pass over the new tokens' q, k and v. A lane owns an octet (8
// consecutive dims, one 16-byte load); D/8 lanes form a vector, the key and the
// value vector of a token and head sit side by side in one warp, so the rotation
// partner of half-split pairs, a group's absmax (4 lanes) and the marking of a
// token with a non-finite value are warp shuffles and a ballot. A lane's 8 codes
// are one 32-bit word of the packed vector.
//
// Per token 2 (Hq + 2 Hkv) D bytes in, 2 Hq D + Hkv (D + D/8) out; the rotation
// row (4 D bytes) is read by every head of a token, so from L1.
// Measured (20 query, 5 key/value heads of 128): 6 x 2048 tokens 44.8 us with cold
// caches, 3.9 TB/s of rows and codes, 80% of the issue slots: the quantisation's
// arithmetic is the bound above a few thousand tokens, two dependent look-ups (the
// token's sequence, its page) below: 64 tokens 2.7 us.
#include "kv4.cuh"

namespace bl {
namespace {

constexpr int kThreads = 256;
// Below: one step a warp, so that the look-ups overlap. Append of 64 tokens 2.7 us against 3.8 with five steps, 256
// tokens 4.4 and 5.0; 384 tokens 6.1 and 5.9, 2048 of one sequence 12.4 and 8.8. Read: 2.1 and 2.3, 3.4 and 3.6, 4.3 and
// 4.4, 3.3 and 2.8 (20 query and 5 key/value heads of 128).
constexpr int64_t kFewTokens = 384;

struct AppendArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, qo_stride;
    uint16_t* q_out;
    const float* cos_sin;
    int64_t max_pos;
    Kv4View cache;
    Kv4Seqs batch;
    int M, Hq;
    int interleaved;
    unsigned* err;
};

__device__ __forceinline__ void unpack_octet(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

// The rotation of a lane's octet `o` (dims 8 o ..): r = fl(fl(x c) + fl(partner s)), with the sign of the
// partner's product in s (a product's rounding does not depend on its sign).
struct Turn {
    float c[8], s[8];
};

template <int D>
__device__ __forceinline__ Turn load_turn(const float* row, int o, bool interleaved) {
    Turn t;
    if (interleaved) {  // pair j of the octet: entry 4 o + j, for both of its dims
        const float4 c = *reinterpret_cast<const float4*>(row + 4 * o), s = *reinterpret_cast<const float4*>(row + D / 2 + 4 * o);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) t.c[2 * j] = t.c[2 * j + 1] = cc[j], t.s[2 * j] = -ss[j], t.s[2 * j + 1] = ss[j];
        return t;
    }
    const int i = 8 * (o & (D / 16 - 1));
    const bool low = o < D / 16;  // the octet holds the a of its pairs
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 c = *reinterpret_cast<const float4*>(row + i + 4 * h), s = *reinterpret_cast<const float4*>(row + D / 2 + i + 4 * h);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) t.c[4 * h + j] = cc[j], t.s[4 * h + j] = low ? -ss[j] : ss[j];
    }
    return t;
}

// Rotate an octet of a vector held by D/8 adjacent lanes. Every lane of the warp calls it.
template <int D>
__device__ __forceinline__ void rotate_octet(const uint4& raw, const Turn& t, bool interleaved, float (&r)[8]) {
    float x[8], p[8];
    unpack_octet(raw, x);
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = x[j ^ 1];
    } else {
        uint4 other;
        other.x = __shfl_xor_sync(0xffffffffu, raw.x, D / 16);
        other.y = __shfl_xor_sync(0xffffffffu, raw.y, D / 16);
        other.z = __shfl_xor_sync(0xffffffffu, raw.z, D / 16);
        other.w = __shfl_xor_sync(0xffffffffu, raw.w, D / 16);
        unpack_octet(other, p);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = __fadd_rn(__fmul_rn(x[j], t.c[j]), __fmul_rn(p[j], t.s[j]));
}

// Threads (x, m): warps of token m. A warp takes STEPS times 32 octets: with several steps the search for the
// token's sequence and the rotation row (a lane's octet of a vector is the same in every step) are shared, with
// one step there are the most warps, for few tokens.
template <int D, int STEPS>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const AppendArgs a) {
    constexpr int LPV = D / 8;  // lanes of a vector
    constexpr int G = D / kKvGroup;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, m = blockIdx.y * blockDim.y + threadIdx.y;
    // octets first + stride st of the token: every warp has its share of the keys and values, which cost more
    const int first = (int)(blockIdx.x * blockDim.x + threadIdx.x), stride = (int)(gridDim.x * blockDim.x);

    if (m >= a.M) return;
    const int kv_lanes = 2 * LPV * a.cache.hkv, all_lanes = kv_lanes + LPV * a.Hq;
    const int o = lane % LPV;  // octet of the vector
    const int g = o >> 2, t = o & 3;
    const bool is_v = (lane / LPV) & 1;  // of the key and value octets: 32 is a multiple of 2 LPV
    const uint16_t* kv = (is_v ? a.v + m * a.v_stride : a.k + m * a.k_stride) + 8 * o;
    const uint16_t* q = a.q + m * a.q_stride + 8 * o;
    uint4 raw[STEPS];  // under way while the token's place is looked up
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
        const int item = first + stride * st;
        raw[st] = make_uint4(0, 0, 0, 0);
        if (item < kv_lanes)
            raw[st] = *reinterpret_cast<const uint4*>(kv + item / (2 * LPV) * D);
        else if (item < all_lanes)
            raw[st] = *reinterpret_cast<const uint4*>(q + (item - kv_lanes) / LPV * D);
    }
    const int s = kv4_seq_of_row(a.batch, m);
    if (s >= a.batch.S) return;  // padding
    const int n_end = a.batch.q_start[s + 1], len = a.batch.kv_len[s];
    const int64_t pos = (int64_t)len - n_end + m;
    if (len < 0 || m < a.batch.q_start[s] || n_end > a.M || pos >= a.max_pos ||
        pos >= ((int64_t)a.batch.W << a.cache.page_shift)) {
        if (lane == 0) atomicOr(a.err, kErrBadBatch);
        return;
    }
    if (pos < 0) return;  // no place in the cache: padding of an idle sequence
    const bool interleaved = a.interleaved != 0;
    const Turn turn = load_turn<D>(a.cos_sin + pos * D, o, interleaved);
    int64_t at = 0;  // this token's vector of head 0
    if (first < kv_lanes) {
        at = kv4_vector(a.cache, a.batch, s, (int)pos, 0);
        if (at < 0) atomicOr(a.err, kErrBadBatch);
    }
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
        const int item = first + stride * st;
        const bool is_kv = item < kv_lanes;
        float x[8];
        rotate_octet<D>(raw[st], turn, interleaved, x);
        if (!is_kv && item < all_lanes)
            *reinterpret_cast<uint4*>(a.q_out + m * a.qo_stride + (item - kv_lanes) / LPV * D + 8 * o) =
                make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        if (!__any_sync(0xffffffffu, is_kv)) continue;
        if (is_v) unpack_octet(raw[st], x);
        float top = fabsf(x[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) top = max_nan(top, fabsf(x[j]));
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const unsigned votes = __ballot_sync(0xffffffffu, !(top < kKvHuge) && is_kv);
        if (is_kv && at >= 0) {
            // the key and value lanes of this token and head
            const bool marked = (votes & (LPV == 16 ? 0xffffffffu : 0xffffu << (lane & 16))) != 0;
            const float step = marked ? 0.0f : kv4_step(top);
            const uint32_t word = step > 0.0f ? kv4_word(x, step) : 0x88888888u;
            const int64_t vec = at + ((int64_t)(item / (2 * LPV)) << a.cache.page_shift);
            *reinterpret_cast<uint32_t*>((is_v ? a.cache.vc : a.cache.kc) + vec * (D / 2) + 4 * (t * G + g)) = word;
            if (t == 0)
                (is_v ? a.cache.vs : a.cache.ks)[vec * G + g] =
                    marked && !is_v ? (uint16_t)0x7FC0 : (uint16_t)(__float_as_uint(step) >> 16);
        }
        __syncwarp();
    }
}

// Blocks of at most 8 warps: x the warps of a token, y tokens (a single warp a token is too small a block).
struct Shape {
    dim3 grid, block;
};
Shape shape_of(int warps, int64_t M, bool one_token) {
    const int x = warps < kThreads / 32 ? warps : kThreads / 32, y = one_token ? 1 : kThreads / 32 / x;
    return {dim3((unsigned)((warps + x - 1) / x), (unsigned)((M + y - 1) / y)), dim3(32 * x, y)};
}

template <int D, int STEPS>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
    const int octets = (2 * a.cache.hkv + a.Hq) * (D / 8);
    const int warps = (octets + 32 * STEPS - 1) / (32 * STEPS);
    const Shape g = shape_of(warps, a.M, true);
    return launch_pdl(kv4_append_kernel<D, STEPS>, g.grid, g.block, 0, s, a);
}

// Threads (x, m): octets of token m, one a lane; a warp takes STEPS times 32.
template <int D, int STEPS>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4View cache, const Kv4Seqs batch, int M, uint16_t* k,
                                                            uint16_t* v, unsigned* err) {
    constexpr int LPV = D / 8;
    constexpr int G = D / kKvGroup;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, m = blockIdx.y * blockDim.y + threadIdx.y;
    const int first = (int)(blockIdx.x * blockDim.x + threadIdx.x - lane) * STEPS + lane;
    if (m >= M) return;
    const int s = kv4_seq_of_row(batch, m);
    if (s >= batch.S) return;
    const int n_end = batch.q_start[s + 1], len = batch.kv_len[s];
    const int64_t pos = (int64_t)len - n_end + m;
    if (len < 0 || m < batch.q_start[s] || n_end > M || pos >= ((int64_t)batch.W << cache.page_shift)) {
        if (lane == 0) atomicOr(err, kErrBadBatch);
        return;
    }
    if (pos < 0) return;
    const int64_t at = kv4_vector(cache, batch, s, (int)pos, 0);
    if (at < 0) {
        if (lane == 0) atomicOr(err, kErrBadBatch);
        return;
    }
    const int o = lane % LPV, g = o >> 2, t = o & 3;
    const bool is_v = (lane / LPV) & 1;
    const uint8_t* codes = (is_v ? cache.vc : cache.kc) + at * (D / 2) + 4 * (t * G + g);
    const uint16_t* steps = (is_v ? cache.vs : cache.ks) + at * G + g;
    uint16_t* out = (is_v ? v : k) + (int64_t)m * cache.hkv * D + 8 * o;
    const int64_t head_vecs = (int64_t)1 << cache.page_shift;
    uint32_t w[STEPS], st[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int head = (first + 32 * i) / (2 * LPV);
        if (head < cache.hkv) {
            w[i] = *reinterpret_cast<const uint32_t*>(codes + head * head_vecs * (D / 2));
            st[i] = steps[head * head_vecs * G];
        }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int head = (first + 32 * i) / (2 * LPV);
        if (head >= cache.hkv) return;
        const uint32_t ss = st[i] | st[i] << 16;
        const uint32_t s16 = bf16x2_mul(ss, kBf16x2Sixteen), s24 = bf16x2_mul(ss, kBf16x2MinusTwentyFour);
        uint32_t p[4];  // pairs (i, i + 4)
        p[0] = bf16x2_fma(kv4_unit_pair<0>(w[i]), s16, s24);
        p[1] = bf16x2_fma(kv4_unit_pair<1>(w[i]), s16, s24);
        p[2] = bf16x2_fma(kv4_unit_pair<2>(w[i]), s16, s24);
        p[3] = bf16x2_fma(kv4_unit_pair<3>(w[i]), s16, s24);
        *reinterpret_cast<uint4*>(out + head * D) =
            make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410), __byte_perm(p[0], p[1], 0x7632),
                       __byte_perm(p[2], p[3], 0x7632));
    }
}

template <int D, int STEPS>
cudaError_t launch_read(const Kv4View& cache, const Kv4Seqs& batch, int64_t M, uint16_t* k, uint16_t* v, unsigned* err,
                        cudaStream_t s) {
    const int warps = (2 * cache.hkv * (D / 8) + 32 * STEPS - 1) / (32 * STEPS);
    const Shape g = shape_of(warps, M, false);
    return launch_pdl(kv4_read_kernel<D, STEPS>, g.grid, g.block, 0, s, cache, batch, (int)M, k, v, err);
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, int64_t M, int Hq, int D, const float* cos_sin, int64_t max_pos,
                              int interleaved, const Kv4View& cache, const Kv4Seqs& batch, uint16_t* q_out,
                              int64_t qo_stride, cudaStream_t s) {
    AppendArgs a;
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.qo_stride = qo_stride;
    a.q_out = q_out, a.cos_sin = cos_sin, a.max_pos = max_pos;
    a.cache = cache, a.batch = batch;
    a.M = (int)M, a.Hq = Hq, a.interleaved = interleaved;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    const bool few = M < kFewTokens;
    if (D == 128) return few ? launch_append<128, 1>(a, s) : launch_append<128, 5>(a, s);
    return few ? launch_append<64, 1>(a, s) : launch_append<64, 5>(a, s);
}

cudaError_t launch_kv4_read(const Kv4View& cache, const Kv4Seqs& batch, int64_t M, int D, uint16_t* k, uint16_t* v,
                            cudaStream_t s) {
    unsigned* err = nullptr;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    const bool few = M < kFewTokens;
    if (D == 128) return few ? launch_read<128, 1>(cache, batch, M, k, v, err, s) : launch_read<128, 5>(cache, batch, M, k, v, err, s);
    return few ? launch_read<64, 1>(cache, batch, M, k, v, err, s) : launch_read<64, 5>(cache, batch, M, k, v, err, s);
}

}  // namespace bl
