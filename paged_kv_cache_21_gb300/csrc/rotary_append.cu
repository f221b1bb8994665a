// kv_append_rotary, kv_latent_append, kv_rotary_frequencies: queries and keys turned by
// their positions on the way into the query buffer and the paged caches.
//
// Both kernels stream: each input is read once, in 16-byte pieces, each output written
// once.  A warp has a token: it works out the token's angles together, an angle a lane and
// step, and its lanes then go over the heads' units (16 elements, eight pairs: rotary.cuh)
// with four units' loads under way each.  Few tokens: their heads are shared out over more
// warps, which each work out the angles.  (A thread for each unit with eight angles of its
// own, in doubles, took 57 us for 8192 tokens of 32 + 8 heads; 24 us of FP64.)
//
// On the device (a captured run of calls over sets of buffers that together exceed L2) and a
// call: 8192 tokens, 32 q / 8 KV heads, d128: 32.4 and 32.7 us, HBM, 6.2 TB/s of its 201 MB;
// 256 tokens to E4M3: 5.0 and 8.4, the host; one token: 2.1 and 8.0.  Latent rows of 512 + 64
// and 16 heads, 8192 tokens: 12.5 and 14.7 to 17.8, for 7.9 at HBM's rate: a token, or four of
// its heads, a warp, each a chain of slot, loads, angles and stores with nothing loaded ahead;
// 32 tokens, 128 heads: 2.5 and 12.5 to 13.5, the host.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>

#include "device_common.cuh"
#include "internal.h"
#include "paged_kv.h"
#include "rotary.cuh"
#include "tree_common.cuh"

namespace pkv {

__device__ DevErr g_rotary_err;
static Launched g_launched;

namespace {

constexpr int kThreads = 128;
constexpr int kCtas = 5;                 // of an SM

constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 256;             // elements of a head that are turned, at most
constexpr int kAhead = 4;                // units whose loads a lane has under way

struct RotaryParams {
    const uint16_t* x[3];                // q, k, v: [T] rows of heads, D elements each
    long long stride[3];                 // elements from one token to the next
    uint16_t* q_out;
    long long out_stride;
    uint8_t* cache[2];                   // K, V
    const int64_t* slots;
    const int64_t* positions;
    const float* inv_freq;
    long long num_slots;
    int T, Hq, Hkv, D, rot, units, share;        // share: warps of a token
    float magnitude, k_scale, v_scale;
};

// The heads are q's, then k's, then v's; a warp's lanes take 32 / units heads at a time, a
// unit each.
template <bool FP8, bool INTER>
__global__ void __launch_bounds__(kThreads, kCtas) kv_append_rotary_kernel(const __grid_constant__ RotaryParams p)
{
    __shared__ __align__(16) float s_cos[kWarps][kMaxDim / 2], s_sin[kWarps][kMaxDim / 2];     // (rotary_take: by fours)
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * kWarps + warp;
    const long long t = job / p.share;
    if (t >= p.T) return;
    const int64_t pos = __ldg(p.positions + t);
    const long long slot = __ldg(p.slots + t);
    const int per = 32 / p.units, u = lane % p.units, first = lane / p.units;    // heads at a time
    const int part = (int)(job - t * p.share), heads = p.Hq + 2 * p.Hkv, step = per * p.share;
    int a, b;
    rotary_pieces(u, p.rot, INTER, a, b);
    const bool turned = u * kRotaryUnit < p.rot;
    auto which = [&](int h) { return h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2; };
    auto within = [&](int h, int w) { return h - (w == 0 ? 0 : w == 1 ? p.Hq : p.Hq + p.Hkv); };
    uint4 xa[kAhead], xb[kAhead];
    int h0 = first < per ? part * per + first : heads;
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int h = h0 + k * step;
            if (h >= heads) continue;
            const int w = which(h);
            const uint16_t* src = p.x[w] + t * p.stride[w] + (long long)within(h, w) * p.D;
            xa[k] = *reinterpret_cast<const uint4*>(src + a);
            xb[k] = *reinterpret_cast<const uint4*>(src + b);
        }
    };
    load();                              // (on their way while the angles are worked out)
    rotary_table(p.inv_freq, p.rot / 2, pos, p.magnitude, s_cos[warp], s_sin[warp], lane);
    float c[8], s[8];
    if (turned) rotary_take(s_cos[warp], s_sin[warp], u, c, s);
    const bool live = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && lane == 0 && part == 0) raise_flag(&g_rotary_err, KV_DEVERR_SLOT_OUT_OF_RANGE, slot);
    const long long blk = slot >> 4, off = slot & 15;
    while (h0 < heads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int h = h0 + k * step;
            if (h >= heads) continue;
            const int w = which(h), hh = within(h, w);
            float y[16];
            const bool turn = turned && w < 2;
            if (turn) {
                float x[16];
                unpack8(xa[k], x);
                unpack8(xb[k], x + 8);
                rotary_turn(x, c, s, INTER, y);
            }
            if (w == 0) {
                uint16_t* dst = p.q_out + t * p.out_stride + (long long)hh * p.D;
                *reinterpret_cast<uint4*>(dst + a) = turn ? pack8(y) : xa[k];
                *reinterpret_cast<uint4*>(dst + b) = turn ? pack8(y + 8) : xb[k];
                continue;
            }
            if (!live) continue;
            uint8_t* cache = p.cache[w - 1];
            const long long at = ((blk * p.Hkv + hh) * kBlock + off) * p.D;
            if (!FP8) {
                *reinterpret_cast<uint4*>(cache + (at + a) * 2) = turn ? pack8(y) : xa[k];
                *reinterpret_cast<uint4*>(cache + (at + b) * 2) = turn ? pack8(y + 8) : xb[k];
            } else {
                // (a turned key goes to its code from binary32, without a rounding to bf16)
                const float scale = w == 1 ? p.k_scale : p.v_scale;
                *reinterpret_cast<uint2*>(cache + at + a) = turn ? quantize8_f32(y, scale) : quantize8_e4m3(xa[k], scale);
                *reinterpret_cast<uint2*>(cache + at + b) = turn ? quantize8_f32(y + 8, scale) : quantize8_e4m3(xb[k], scale);
            }
        }
        h0 += kAhead * step;
        load();
    }
}

// ------------------------------------------------------------------ latent

struct LatentAppendParams {
    const uint16_t* latent;
    const uint16_t* k_rope;
    const uint16_t* weight;              // bf16 [L], or null: no norm
    const uint16_t* q;
    uint16_t* q_out;
    uint16_t* cache;                     // [slots][L + R]
    const int64_t* slots;
    const int64_t* positions;
    const float* inv_freq;
    long long latent_stride, rope_stride, q_token, q_head, out_token, out_head, num_slots;
    int T, H, L, R, share;               // share: warps of a token's queries
    int row_blocks;                      // CTAs that write cache rows, a warp a token; the others turn queries
    float eps, magnitude;
};

constexpr int kLatentCtas = 8;           // of an SM: little work a warp, so many warps (8192 tokens: 12.4 us, with 5 or 6 12.9)
constexpr int kLatentAhead = 2;
constexpr int kLatentMax = 1024;         // elements of a latent vector

template <bool INTER>
__global__ void __launch_bounds__(kThreads, kLatentCtas) kv_latent_append_kernel(const __grid_constant__ LatentAppendParams p)
{
    __shared__ __align__(16) float s_cos[kWarps][kMaxDim / 2], s_sin[kWarps][kMaxDim / 2];     // (rotary_take: by fours)
    pdl_wait();
    const int units = p.R / kRotaryUnit, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* cs = s_cos[warp];
    float* sn = s_sin[warp];
    if ((int)blockIdx.x < p.row_blocks) {
        const long long t = (long long)blockIdx.x * kWarps + warp;
        if (t >= p.T) return;
        const int64_t pos = __ldg(p.positions + t);
        const long long slot = __ldg(p.slots + t);
        // the latent vector: 16-byte pieces lane, lane + 32, ...; the key part: a lane a unit
        constexpr int kPieces = kLatentMax / 256;
        uint4 v[kPieces], xa, xb;
        const uint16_t* src = p.latent + t * p.latent_stride;
        const uint16_t* kr = p.k_rope + t * p.rope_stride;
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            if ((lane + 32 * k) * 8 < p.L) v[k] = *reinterpret_cast<const uint4*>(src + (lane + 32 * k) * 8);
        int a, b;
        rotary_pieces(lane, p.R, INTER, a, b);
        if (lane < units) {
            xa = *reinterpret_cast<const uint4*>(kr + a);
            xb = *reinterpret_cast<const uint4*>(kr + b);
        }
        if (slot < 0) return;                             // padding token
        if (slot >= p.num_slots) {
            if (lane == 0) raise_flag(&g_rotary_err, KV_DEVERR_SLOT_OUT_OF_RANGE, slot);
            return;
        }
        uint16_t* row = p.cache + slot * (p.L + p.R);
        rotary_table(p.inv_freq, p.R / 2, pos, p.magnitude, cs, sn, lane);
        if (lane < units) {
            float x[16], y[16], c[8], s[8];
            rotary_take(cs, sn, lane, c, s);
            unpack8(xa, x);
            unpack8(xb, x + 8);
            rotary_turn(x, c, s, INTER, y);
            *reinterpret_cast<uint4*>(row + p.L + a) = pack8(y);
            *reinterpret_cast<uint4*>(row + p.L + b) = pack8(y + 8);
        }
        if (!p.weight) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                if ((lane + 32 * k) * 8 < p.L) *reinterpret_cast<uint4*>(row + (lane + 32 * k) * 8) = v[k];
            return;
        }
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            if ((lane + 32 * k) * 8 >= p.L) continue;
            float x[8];
            unpack8(v[k], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        const float inv = 1.f / sqrtf(sum / (float)p.L + p.eps);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int at = (lane + 32 * k) * 8;
            if (at >= p.L) continue;
            float x[8], w[8];
            unpack8(v[k], x);
            unpack8(__ldg(reinterpret_cast<const uint4*>(p.weight + at)), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
            *reinterpret_cast<uint4*>(row + at) = pack8(x);
        }
        return;
    }
    // ---- queries: a warp's lanes take 32 / units heads at a time, a unit each
    const long long job = (long long)(blockIdx.x - p.row_blocks) * kWarps + warp;
    const long long t = job / p.share;
    if (t >= p.T) return;
    const int64_t pos = __ldg(p.positions + t);
    const int per = 32 / units, u = lane % units, first = lane / units;
    const int part = (int)(job - t * p.share), step = per * p.share;
    int a, b;
    rotary_pieces(u, p.R, INTER, a, b);
    uint4 xa[kLatentAhead], xb[kLatentAhead];
    int h0 = first < per ? part * per + first : p.H;
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kLatentAhead; ++k) {
            const int h = h0 + k * step;
            if (h >= p.H) continue;
            const uint16_t* src = p.q + t * p.q_token + h * p.q_head;
            xa[k] = *reinterpret_cast<const uint4*>(src + a);
            xb[k] = *reinterpret_cast<const uint4*>(src + b);
        }
    };
    load();                              // (on their way while the angles are worked out)
    rotary_table(p.inv_freq, p.R / 2, pos, p.magnitude, cs, sn, lane);
    float c[8], s[8];
    rotary_take(cs, sn, u, c, s);
    while (h0 < p.H) {
#pragma unroll
        for (int k = 0; k < kLatentAhead; ++k) {
            const int h = h0 + k * step;
            if (h >= p.H) continue;
            float x[16], y[16];
            unpack8(xa[k], x);
            unpack8(xb[k], x + 8);
            rotary_turn(x, c, s, INTER, y);
            uint16_t* dst = p.q_out + t * p.out_token + h * p.out_head;
            *reinterpret_cast<uint4*>(dst + a) = pack8(y);
            *reinterpret_cast<uint4*>(dst + b) = pack8(y + 8);
        }
        h0 += kLatentAhead * step;
        load();
    }
}

// Warps of a token: one where the tokens fill the device, more where they do not, but no
// more than there are steps of its heads.
int warps_of_token(int tokens, int heads, int heads_at_a_time, int ctas)
{
    const long long want = (long long)num_sms_current() * ctas * kWarps;
    const long long s = (want + tokens - 1) / tokens, most = (heads + heads_at_a_time - 1) / heads_at_a_time;
    return (int)(s < 1 ? 1 : s > most ? most : s);
}

template <typename P>
int launch(void (*kernel)(const P), long long blocks, const P& p, void* stream)
{
    if (blocks > INT32_MAX) return KV_ERR_UNSUPPORTED;
    g_launched.note();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

bool aligned16(std::initializer_list<const void*> ptrs)
{
    uintptr_t any = 0;
    for (const void* x : ptrs) any |= (uintptr_t)x;
    return (any & 15) == 0;
}

// Is `stride`, in elements of two bytes, one that 16-byte accesses can take?
bool good_stride(int64_t stride, int64_t least) { return stride >= least && stride % 8 == 0; }

}  // namespace

int rotary_read_error(unsigned* flags, long long* detail) { return g_launched.take_error(g_rotary_err, flags, detail); }

}  // namespace pkv

using namespace pkv;

extern "C" int kv_append_rotary(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride,
                                const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                void* k_cache, void* v_cache, const int64_t* slot_mapping,
                                const int64_t* positions, const float* inv_freq, int rotary_dim,
                                unsigned flags, float magnitude, int num_tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, int num_blocks, int kv_dtype,
                                float k_scale, float v_scale, void* stream)
{
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_blocks <= 0 || head_dim <= 0 ||
        rotary_dim <= 0 || rotary_dim > head_dim || (flags & ~KV_ROTARY_INTERLEAVED) || !std::isfinite(magnitude))
        return KV_ERR_INVALID_ARG;
    if (head_dim % kRotaryUnit || rotary_dim % kRotaryUnit || head_dim > 32 * kRotaryUnit || rotary_dim > kMaxDim)
        return KV_ERR_UNSUPPORTED;
    if (kv_dtype != KV_DTYPE_BF16 && kv_dtype != KV_DTYPE_FP8_E4M3) return KV_ERR_UNSUPPORTED;
    const int64_t qrow = (int64_t)num_q_heads * head_dim, kvrow = (int64_t)num_kv_heads * head_dim;
    if (qrow > INT32_MAX / 4 || kvrow > INT32_MAX / 4) return KV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return KV_OK;
    if (!k || !v || !k_cache || !v_cache || !slot_mapping || !positions || !inv_freq) return KV_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!q || !q_out)) return KV_ERR_INVALID_ARG;
    if (!aligned16({q, q_out, k, v, k_cache, v_cache})) return KV_ERR_INVALID_ARG;
    if (!good_stride(k_stride, kvrow) || !good_stride(v_stride, kvrow)) return KV_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!good_stride(q_stride, qrow) || !good_stride(q_out_stride, qrow)))
        return KV_ERR_INVALID_ARG;
    const bool fp8 = kv_dtype == KV_DTYPE_FP8_E4M3;
    if (fp8 && !(k_scale > 0.f && v_scale > 0.f && std::isfinite(k_scale) && std::isfinite(v_scale)))
        return KV_ERR_INVALID_ARG;
    RotaryParams p;
    p.x[0] = static_cast<const uint16_t*>(q);
    p.x[1] = static_cast<const uint16_t*>(k);
    p.x[2] = static_cast<const uint16_t*>(v);
    p.stride[0] = q_stride;
    p.stride[1] = k_stride;
    p.stride[2] = v_stride;
    p.q_out = static_cast<uint16_t*>(q_out);
    p.out_stride = q_out_stride;
    p.cache[0] = static_cast<uint8_t*>(k_cache);
    p.cache[1] = static_cast<uint8_t*>(v_cache);
    p.slots = slot_mapping;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.num_slots = (long long)num_blocks * kBlock;
    p.T = num_tokens;
    p.Hq = num_q_heads;
    p.Hkv = num_kv_heads;
    p.D = head_dim;
    p.rot = rotary_dim;
    p.units = head_dim / kRotaryUnit;
    p.share = warps_of_token(num_tokens, num_q_heads + 2 * num_kv_heads, 32 / p.units, kCtas);
    p.magnitude = magnitude;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    const long long blocks = ((long long)num_tokens * p.share + kWarps - 1) / kWarps;
    const bool inter = flags & KV_ROTARY_INTERLEAVED;
    auto* kernel = fp8 ? (inter ? kv_append_rotary_kernel<true, true> : kv_append_rotary_kernel<true, false>)
                       : (inter ? kv_append_rotary_kernel<false, true> : kv_append_rotary_kernel<false, false>);
    return launch(kernel, blocks, p, stream);
}

extern "C" int kv_latent_append(void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                                const void* q_rope, int64_t q_token_stride, int64_t q_head_stride,
                                const void* latent, int64_t latent_stride, const void* k_rope,
                                int64_t k_rope_stride, const void* norm_weight, float eps, void* cache,
                                const int64_t* slot_mapping, const int64_t* positions,
                                const float* inv_freq, unsigned flags, float magnitude, int num_tokens,
                                int num_q_heads, int latent_dim, int rope_dim, int num_blocks,
                                void* stream)
{
    if (num_tokens < 0 || num_q_heads < 0 || latent_dim <= 0 || rope_dim <= 0 || num_blocks <= 0 ||
        (flags & ~KV_ROTARY_INTERLEAVED) || !std::isfinite(magnitude))
        return KV_ERR_INVALID_ARG;
    if (latent_dim % 8 || latent_dim > kLatentMax || rope_dim % kRotaryUnit || rope_dim > kMaxDim)
        return KV_ERR_UNSUPPORTED;
    if ((int64_t)num_q_heads * rope_dim > INT32_MAX / 4) return KV_ERR_UNSUPPORTED;
    if (norm_weight && !(eps >= 0.f && std::isfinite(eps))) return KV_ERR_INVALID_ARG;
    if (num_tokens == 0) return KV_OK;
    if (!latent || !k_rope || !cache || !slot_mapping || !positions || !inv_freq) return KV_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!q_rope || !q_out)) return KV_ERR_INVALID_ARG;
    if (!aligned16({q_out, q_rope, latent, k_rope, norm_weight, cache})) return KV_ERR_INVALID_ARG;
    if (!good_stride(latent_stride, latent_dim) || !good_stride(k_rope_stride, rope_dim)) return KV_ERR_INVALID_ARG;
    if (num_q_heads > 0) {
        // (heads apart by a row at least, tokens by all their heads: no element is written twice)
        if (!good_stride(q_head_stride, rope_dim) || !good_stride(q_out_head_stride, rope_dim) ||
            q_head_stride > INT64_MAX / 2 / num_q_heads || q_out_head_stride > INT64_MAX / 2 / num_q_heads)
            return KV_ERR_INVALID_ARG;
        const int64_t last = num_q_heads - 1;
        if (!good_stride(q_token_stride, last * q_head_stride + rope_dim) ||
            !good_stride(q_out_token_stride, last * q_out_head_stride + rope_dim))
            return KV_ERR_INVALID_ARG;
    }
    LatentAppendParams p;
    p.latent = static_cast<const uint16_t*>(latent);
    p.k_rope = static_cast<const uint16_t*>(k_rope);
    p.weight = static_cast<const uint16_t*>(norm_weight);
    p.q = static_cast<const uint16_t*>(q_rope);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.cache = static_cast<uint16_t*>(cache);
    p.slots = slot_mapping;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.latent_stride = latent_stride;
    p.rope_stride = k_rope_stride;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.out_token = q_out_token_stride;
    p.out_head = q_out_head_stride;
    p.num_slots = (long long)num_blocks * kBlock;
    p.T = num_tokens;
    p.H = num_q_heads;
    p.L = latent_dim;
    p.R = rope_dim;
    p.eps = eps;
    p.magnitude = magnitude;
    const int units = rope_dim / kRotaryUnit;
    p.row_blocks = (num_tokens - 1) / kWarps + 1;
    p.share = num_q_heads > 0 ? warps_of_token(num_tokens, num_q_heads, 32 / units, kLatentCtas) : 0;
    const long long blocks = p.row_blocks + ((long long)num_tokens * p.share + kWarps - 1) / kWarps;
    return launch(flags & KV_ROTARY_INTERLEAVED ? kv_latent_append_kernel<true> : kv_latent_append_kernel<false>, blocks,
                  p, stream);
}

extern "C" int kv_rotary_frequencies(float* inv_freq, float* magnitude, int rotary_dim, double theta,
                                     int scaling, double factor, double low, double high,
                                     double original_len)
{
    if (!inv_freq || rotary_dim <= 0 || rotary_dim % 2 || !(theta > 0.0) || !std::isfinite(theta))
        return KV_ERR_INVALID_ARG;
    if (scaling < KV_ROTARY_PLAIN || scaling > KV_ROTARY_BANDS) return KV_ERR_INVALID_ARG;
    if (scaling != KV_ROTARY_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return KV_ERR_INVALID_ARG;
    const bool parts = scaling == KV_ROTARY_PARTS || scaling == KV_ROTARY_BANDS;
    if (parts && !(low > 0.0 && high > low && std::isfinite(high) && original_len > 0.0 && std::isfinite(original_len)))
        return KV_ERR_INVALID_ARG;
    if (scaling == KV_ROTARY_PARTS && !(theta > 1.0)) return KV_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586477, d = rotary_dim;
    if (scaling == KV_ROTARY_BASE) {
        if (rotary_dim < 4) return KV_ERR_INVALID_ARG;
        theta *= std::pow(factor, d / (d - 2.0));
    }
    // KV_ROTARY_PARTS: the pair that makes `turns` turns over the original length
    auto pair_of = [&](double turns) {
        return d * std::log(original_len / (turns * two_pi)) / (2.0 * std::log(theta));
    };
    double first = 0.0, last = 0.0;
    if (scaling == KV_ROTARY_PARTS) {
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = std::fmin(std::ceil(pair_of(low)), d - 1.0);
        if (last <= first) last = first + 0.001;
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(theta, -2.0 * i / d);
        double g = f;
        if (scaling == KV_ROTARY_LINEAR) {
            g = f / factor;
        } else if (scaling == KV_ROTARY_PARTS) {
            const double slow = std::fmin(std::fmax((i - first) / (last - first), 0.0), 1.0);
            g = f * (1.0 - slow) + f / factor * slow;
        } else if (scaling == KV_ROTARY_BANDS) {
            const double turns = original_len * f / two_pi;
            const double fast = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
            g = f * fast + f / factor * (1.0 - fast);
        }
        inv_freq[i] = (float)g;
    }
    if (magnitude) *magnitude = scaling == KV_ROTARY_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return KV_OK;
}
