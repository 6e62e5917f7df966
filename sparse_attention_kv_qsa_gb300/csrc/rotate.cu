// Rotation of heads by position, alone (rotate) and on the way into a paged
// cache (append).
//
//   pair p of token t's head: (a, b) -> (a cos - b sin, b cos + a sin),  angle = position[axis_p][t] freq_p
//
// What bounds it: every row is read and written once, so HBM; a single token's
// call is launch and latency.
//
// Angles. freq / 2 pi is held in 64-bit fixed point (turns), and position times
// that modulo 2^64 is the angle's fraction of a turn without any error but the
// factor's own (2^-64 of the position, for every frequency): whole turns fall off by themselves at
// every position. The nearest quarter turn is split off, so that sine and
// cosine are of at most an eighth, in fp32.
//
// Work. A row is a token's head. 16 lanes (a team) take a row, 8 elements each;
// a CTA has 8 or 16 teams and a power of two of tokens, every team rows of one token
// alone, so that a lane's 8 sines and cosines stay in registers. They are found
// once per token by 64 threads, through shared memory. Rows are read ahead, three or four
// per team, before anything that has to be looked up (the token's sequence by a
// 32-way search in cu, its length, its page).
//
// Measured (GB300): 16,384 tokens of 24 bfloat16 heads on three axes 35.2 us, 5.7 TB/s (0.84 of the
// measured copy rate); ragged prompts of 20,797 tokens appended, 32 query heads on 8, 99 us, 5.6 TB/s (0.82);
// 256 single tokens of 72 rows 5.8 us and one of 48 rows 3.3 us on the device, where the chain sequence - length -
// page and one barrier are what counts, and where a token has more rows than are ahead a second round of loads; 4,192 tokens
// to int8 cells 33 us, three waves of CTAs of the same chain with four rounds of loads each.
#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "cache_internal.cuh"
#include "ptx.cuh"
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int FEW_TOKENS_THREADS = 256, MANY_TOKENS_THREADS = 128;
constexpr int LANES = 16;
constexpr int MAX_PAIRS = 64;
constexpr int NO_PAGES = -1;

struct Params {
    const void *src[3];                  // keys, values, then queries (rotate: queries alone)
    int64_t src_tok[3], src_head[3];
    void *q_out, *k_out;
    int64_t q_out_tok, q_out_head, k_out_tok, k_out_head;
    int ntok, nheads, nkv;               // rows of a token: nkv keys, nkv values, nheads queries
    int tokens;                          // of a CTA
    qsa_rotation rot;
    qsa_kv_pages kv;
    const int32_t *table, *lens, *cu;
    int table_cols, nseq;
    int64_t table_stride;
    Divider page;
};

// Where a token's cell lies: element offsets of its page and slot; -1: not written. scale: of the scales.
struct Place {
    int64_t at, scale;
    int cell;                            // position where none is given
    int member;                          // of a sequence
};

template <typename T>
struct Raw {   // 8 elements as they lie
    static constexpr int WORDS = sizeof(T) * 2;
    uint32_t w[WORDS];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_row(const T *p) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < Raw<T>::WORDS / 4; ++i) {
        const uint4 v = ld_in(reinterpret_cast<const uint4 *>(p) + i);
        r.w[4 * i] = v.x;
        r.w[4 * i + 1] = v.y;
        r.w[4 * i + 2] = v.z;
        r.w[4 * i + 3] = v.w;
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void widen(const Raw<T> &r, float (&x)[8]) {
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(r.w[i] << 16);
            x[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
// 8 elements rounded once to T.
template <typename T>
__device__ __forceinline__ void store_row(T *p, const float (&x)[8]) {
    uint32_t w[Raw<T>::WORDS];
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
    }
#pragma unroll
    for (int i = 0; i < Raw<T>::WORDS / 4; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// |freq| / 2 pi in units of 2^-64 turns, modulo a turn, at most 1.01 units too small; the sign goes to the product.
// |freq| = m 2^e has 24 bits m; whole turns of the largest, e = 104, are gone from the 104th bit of 1 / (2 pi) on, and 96
// bits from there give the product's fraction.
__device__ __forceinline__ uint64_t turns_of(float freq) {
    // 2^256 / (2 pi), 64 bits each
    constexpr uint64_t W0 = 0x28be60db9391054aull, W1 = 0x7f09d5f47d4d3770ull, W2 = 0x36d8a5664f10e410ull, W3 = 0x7f9458eaf7aef158ull;
    const uint32_t bits = __float_as_uint(freq), field = (bits >> 23) & 255u;
    const uint32_t m = (bits & 0x7FFFFFu) | (field > 0u ? 0x800000u : 0u);
    const int e = static_cast<int>(max(field, 1u)) - 150;   // |freq| = m 2^e
    uint64_t a = W0, b = W1;                                 // from bit max(e, 0) on
    if (e > 0) {                                             // |freq| of 2^24 at least
        const bool far = e >= 64;
        const int r = e & 63;
        const uint64_t w0 = far ? W1 : W0, w1 = far ? W2 : W1, w2 = far ? W3 : W2;
        a = r == 0 ? w0 : (w0 << r) | (w1 >> (64 - r));
        b = r == 0 ? w1 : (w1 << r) | (w2 >> (64 - r));
    }
    // m (a + b / 2^64) with b's upper half, in 32-bit products: m x 2^-32 of a unit at most is left out.
    const uint64_t p1 = static_cast<uint64_t>(m) * static_cast<uint32_t>(a >> 32);
    const uint64_t p0 = static_cast<uint64_t>(m) * static_cast<uint32_t>(a) + __umulhi(m, static_cast<uint32_t>(b >> 32));
    const uint64_t lo = p0 + (p1 << 32), hi = (p1 + (p0 >> 32)) >> 32;
    uint64_t t;
    if (e >= 0) t = lo;
    else if (e > -64) t = (lo >> -e) | (hi << (64 + e));
    else t = e > -128 ? hi >> (-e - 64) : 0;
    return static_cast<int32_t>(bits) < 0 ? 0 - t : t;
}
// cos and sin of position x turns (a product modulo 2^64).
__device__ __forceinline__ float2 cos_sin(uint64_t turns, int32_t position) {
    const uint32_t u = static_cast<uint32_t>((turns * static_cast<uint64_t>(static_cast<int64_t>(position))) >> 32);
    const uint32_t quarter = (u + 0x20000000u) >> 30;
    const float half_turns = static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * 4.6566128730773926e-10f;   // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    const float a = quarter & 1u ? s : c, b = quarter & 1u ? c : s;
    return make_float2(((quarter + 1u) & 2u) ? -a : a, (quarter & 2u) ? -b : b);
}

// The last sequence that begins at or before token t, found by a whole warp: -1 where t is of none.
__device__ __forceinline__ int sequence_of(const Params &p, int t) {
    const int lane = threadIdx.x & 31;
    int lo = -1, hi = p.nseq + 1;   // cu[lo] <= t < cu[hi], were there such
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, s = lo + (lane + 1) * step;
        const int below = __popc(__ballot_sync(FULL_MASK, s < hi && min(max(ld_in(p.cu + s), 0), p.ntok) <= t));
        lo += below * step;
        hi = min(hi, lo + step);
    }
    return lo == p.nseq ? -1 : lo;
}

// kPages: NO_PAGES (rotate), QSA_BF16, QSA_F16 or QSA_I8.
template <typename T, int kPages, int THREADS>
__global__ void __launch_bounds__(THREADS) rows_kernel(const __grid_constant__ Params p) {
    constexpr bool kAppend = kPages != NO_PAGES;
    constexpr int AHEAD = kPages == QSA_I8 ? 3 : 4;
    constexpr int TEAMS = THREADS / LANES, MAX_TOKENS = TEAMS;
    __shared__ __align__(16) float cosines[MAX_TOKENS][MAX_PAIRS], sines[MAX_TOKENS][MAX_PAIRS];
    __shared__ Place places[MAX_TOKENS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, team = tid / LANES, l = tid % LANES;
    const int t0 = blockIdx.x * p.tokens, mine = team & (p.tokens - 1), t = t0 + mine;
    const int first = team / p.tokens, step = TEAMS / p.tokens;   // tokens: a power of two
    const int rows = 2 * p.nkv + p.nheads;
    const bool turned = p.rot.freqs != nullptr;

    grid_dependency_wait();
    grid_launch_dependents();

    // Row r of the token: its kind (0 key, 1 value, 2 query) and head.
    auto kind = [&](int r, int &h) {
        if (!kAppend || r >= 2 * p.nkv) {
            h = r - 2 * p.nkv;
            return 2;
        }
        h = r < p.nkv ? r : r - p.nkv;
        return r < p.nkv ? 0 : 1;
    };
    Raw<T> raw[AHEAD];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = r0 + i * step;
            int h;
            const int k = kind(r, h);
            if (t < p.ntok && r < rows)
                raw[i] = load_row(static_cast<const T *>(p.src[k]) + t * p.src_tok[k] + h * p.src_head[k] + 8 * l);
            else
#pragma unroll
                for (int e = 0; e < Raw<T>::WORDS; ++e) raw[i].w[e] = 0u;
        }
    };
    load(first);

    // What the angles need comes along with the lookups below.
    const int pair = tid % MAX_PAIRS, i0 = tid / MAX_PAIRS;   // this thread's pair, and first token
    const bool angles = turned && pair < p.rot.npairs;
    float freq = 0.0f;
    bool on_axis = false;
    const int32_t *positions = p.rot.positions;
    int position0 = 0;
    if (angles) {
        freq = ld_in(p.rot.freqs + pair);
        const int axis = p.rot.axis == nullptr ? 0 : ld_in(p.rot.axis + pair);
        on_axis = axis >= 0 && axis < p.rot.naxes;
        if (on_axis && positions != nullptr) {
            positions += axis * p.rot.position_stride + t0;
            if (i0 < p.tokens && t0 + i0 < p.ntok) position0 = ld_in(positions + i0);
        }
    }

    if constexpr (kAppend) {
        for (int i = warp; i < p.tokens; i += THREADS / 32) {
            if (t0 + i >= p.ntok) break;
            const int s = p.cu == nullptr ? t0 + i : sequence_of(p, t0 + i);
            if (lane != 0) continue;
            Place w = {-1, 0, 0, s >= 0};
            if (s >= 0) {
                const int end = p.cu == nullptr ? t0 + i + 1 : min(max(ld_in(p.cu + s + 1), 0), p.ntok);
                w.cell = max(ld_in(p.lens + s), 0) - (end - (t0 + i));
                if (w.cell >= 0 && w.cell < static_cast<long long>(p.table_cols) * p.kv.page_size) {
                    const int column = divide(p.page, w.cell), slot = w.cell - column * p.kv.page_size;
                    const int page = ld_in(p.table + s * p.table_stride + column);
                    if (page >= 0 && page < p.kv.npages) {
                        w.at = page * p.kv.page_stride + slot * p.kv.cell_stride;
                        if constexpr (kPages == QSA_I8) w.scale = page * p.kv.scale_page_stride + slot * p.kv.scale_cell_stride;
                    }
                }
            }
            places[i] = w;
        }
        if (turned && p.rot.positions == nullptr) __syncthreads();   // the same in every thread
    }
    if (angles) {
        const uint64_t turns = on_axis ? turns_of(freq) : 0;
        const float odd = freq * 0.0f;   // NaN where the frequency is not finite
        for (int i = i0; i < p.tokens && t0 + i < p.ntok; i += THREADS / MAX_PAIRS) {
            int position = position0;
            if (kAppend && p.rot.positions == nullptr) position = places[i].cell;
            else if (on_axis && i != i0) position = ld_in(positions + i);
            const float2 cs = cos_sin(turns, position);
            cosines[i][pair] = cs.x + odd;
            sines[i][pair] = (p.rot.inverse ? -cs.y : cs.y) + odd;
        }
    }
    __syncthreads();
    if (__all_sync(FULL_MASK, t >= p.ntok)) return;   // both of the warp's teams

    // This lane's sines and cosines: 8 pairs with the partner in another lane, or 4 of its own.
    const int pairs = p.rot.npairs, apart = pairs / 8;   // lanes between the halves
    const bool own = p.rot.interleaved != 0;
    const bool in_pair = turned && l < 2 * apart;
    const bool second = !own && l >= apart;
    const int partner = in_pair && !own ? (second ? lane - apart : lane + apart) : lane;
    float cosv[8], sinv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cosv[e] = 1.0f;
        sinv[e] = 0.0f;
    }
    if (in_pair) {
        const int from = own ? 4 * l : 8 * (second ? l - apart : l);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (own && e >= 4) break;
            cosv[e] = cosines[mine][from + e];
            sinv[e] = second ? sines[mine][from + e] : -sines[mine][from + e];
        }
    }
    const bool here = t < p.ntok && (!kAppend || places[mine].member != 0);
    for (int r0 = first; r0 - first < rows; r0 += AHEAD * step) {   // as often for both teams of a warp
        if (r0 != first) load(r0);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = r0 + i * step;
            if (r0 - first + i * step >= rows) break;
            float x[8], y[8];
            widen(raw[i], x);
            if (own) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[2 * e] = fmaf(x[2 * e + 1], sinv[e], x[2 * e] * cosv[e]);
                    y[2 * e + 1] = fmaf(x[2 * e], -sinv[e], x[2 * e + 1] * cosv[e]);
                }
            } else {
                Raw<T> other;
#pragma unroll
                for (int e = 0; e < Raw<T>::WORDS; ++e) other.w[e] = __shfl_sync(FULL_MASK, raw[i].w[e], partner);
                float z[8];
                widen(other, z);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fmaf(z[e], sinv[e], x[e] * cosv[e]);
            }
            int h;
            const int k = kind(r, h);
            if (!in_pair || k == 1)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e];
            const bool good = here && r < rows;
            if (k == 2) {
                if (good) store_row(static_cast<T *>(p.q_out) + t * p.q_out_tok + h * p.q_out_head + 8 * l, y);
            } else if (kAppend) {
                if (k == 0 && good && p.k_out != nullptr)
                    store_row(static_cast<T *>(p.k_out) + t * p.k_out_tok + h * p.k_out_head + 8 * l, y);
            }
            if constexpr (kPages == QSA_I8) {
                if (!__any_sync(FULL_MASK, k < 2)) continue;   // queries alone
                // The team's largest magnitude; both teams take part.
                float top = 0.0f, odd = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    top = fmaxf(top, fabsf(y[e]));
                    odd = fmaf(y[e], 0.0f, odd);
                }
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
                const bool bad = (__ballot_sync(FULL_MASK, !(odd == 0.0f)) >> (lane & LANES) & 0xFFFFu) != 0u;
                if (good && k < 2 && places[mine].at >= 0) {
                    const __half scale = __float2half_rn(fminf(__fdiv_rn(top, 127.0f), 65504.0f));
                    const float f = __half2float(scale);
                    uint32_t w[2] = {0u, 0u};
                    if (!bad && f > 0.0f) {
                        // The quotient by the reciprocal is off by less than 2^-15 (of 127 at most, two roundings; near
                        // zero it is cut off all the same): where that could change the nearest integer, divide.
                        const float inv = __frcp_rn(f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float q = y[e] * inv;
                            const float off = fabsf(q - rintf(q));
                            if (!(off < 0.4999f)) q = __fdiv_rn(y[e], f);
                            const int code = min(127, max(-127, __float2int_rn(q)));
                            w[e >> 2] |= (static_cast<uint32_t>(code) & 255u) << (8 * (e & 3));
                        }
                    }
                    int8_t *to = static_cast<int8_t *>(k == 0 ? p.kv.k : p.kv.v) + places[mine].at + h * p.kv.head_stride + 8 * l;
                    *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
                    if (l == 0)
                        (k == 0 ? p.kv.k_scale_f16 : p.kv.v_scale_f16)[places[mine].scale + h * p.kv.scale_head_stride] =
                            bad ? static_cast<uint16_t>(0x7FFF) : __half_as_ushort(scale);
                }
            } else if constexpr (kAppend) {
                using P = typename std::conditional<kPages == QSA_BF16, __nv_bfloat16, __half>::type;
                if (good && k < 2 && places[mine].at >= 0)
                    store_row(static_cast<P *>(k == 0 ? p.kv.k : p.kv.v) + places[mine].at + h * p.kv.head_stride + 8 * l, y);
            }
        }
    }
}

template <typename T, int kPages, int THREADS>
cudaError_t launch_threads(Params p, cudaStream_t stream) {
    // A CTA has some 64 rows (32 of 32 bits) where there are CTAs enough for all SMs. Measured: 16,384 tokens of 24
    // heads 34.9 us, with 32 rows 38.8, with 128 36.3; 4,097 of 16 heads in 32 bits 11.8 us, with 64 rows 13.0.
    const int rows = 2 * p.nkv + p.nheads, wanted = 128 / static_cast<int>(sizeof(T));
    p.tokens = 1;
    while (p.tokens < THREADS / LANES && p.tokens * rows < wanted && p.ntok / p.tokens >= 2 * device_sm_count()) p.tokens *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.ntok + p.tokens - 1) / p.tokens);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rows_kernel<T, kPages, THREADS>, p);
}

// Few tokens' rows are spread over more threads each (one token of 48 rows 3.7 us, with 128 threads 4.3); many tokens'
// CTAs are small, so that more of them are at different stages on an SM (ragged prompts of 48 rows a token 101 us, with 256
// threads 138).
template <typename T, int kPages>
cudaError_t launch(const Params &p, cudaStream_t stream) {
    return p.ntok <= 2 * device_sm_count() ? launch_threads<T, kPages, FEW_TOKENS_THREADS>(p, stream)
                                           : launch_threads<T, kPages, MANY_TOKENS_THREADS>(p, stream);
}

template <typename T>
cudaError_t launch_append_of(const Params &p, cudaStream_t stream) {
    if (p.kv.dtype == QSA_I8) return launch<T, QSA_I8>(p, stream);
    if constexpr (!std::is_same<T, __half>::value)
        if (p.kv.dtype == QSA_BF16) return launch<T, QSA_BF16>(p, stream);
    if constexpr (!std::is_same<T, __nv_bfloat16>::value)
        if (p.kv.dtype == QSA_F16) return launch<T, QSA_F16>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rotate(const void *x, int dtype, const int64_t *strides, int ntok, int nheads, const qsa_rotation &rot,
                          void *out, cudaStream_t stream) {
    Params p = {};
    p.src[2] = x;
    p.src_tok[2] = strides[0];
    p.src_head[2] = strides[1];
    p.q_out = out;
    p.q_out_tok = strides[2];
    p.q_out_head = strides[3];
    p.ntok = ntok;
    p.nheads = nheads;
    p.rot = rot;
    if (dtype == QSA_F32) return launch<float, NO_PAGES>(p, stream);
    return dtype == QSA_F16 ? launch<__half, NO_PAGES>(p, stream) : launch<__nv_bfloat16, NO_PAGES>(p, stream);
}

cudaError_t launch_cache_append(const CacheAppendArgs &a, cudaStream_t stream) {
    Params p = {};
    const void *src[3] = {a.k, a.v, a.q};
    for (int i = 0; i < 3; ++i) {
        p.src[i] = src[i];
        p.src_tok[i] = a.strides[2 * i];
        p.src_head[i] = a.strides[2 * i + 1];
    }
    p.q_out = a.q_out;
    p.q_out_tok = a.strides[6];
    p.q_out_head = a.strides[7];
    p.k_out = a.k_out;
    p.k_out_tok = a.strides[8];
    p.k_out_head = a.strides[9];
    p.ntok = a.ntok;
    p.nheads = a.nheads;
    p.nkv = a.kv.nkv;
    if (a.rotation != nullptr) p.rot = *a.rotation;
    p.kv = a.kv;
    p.table = a.table;
    p.table_cols = a.table_cols;
    p.table_stride = a.table_stride;
    p.lens = a.lens;
    p.cu = a.cu;
    p.nseq = a.nseq;
    p.page = make_divider(a.kv.page_size);
    if (a.dtype == QSA_F32) return launch_append_of<float>(p, stream);
    return a.dtype == QSA_F16 ? launch_append_of<__half>(p, stream) : launch_append_of<__nv_bfloat16>(p, stream);
}

}  // namespace qsa
