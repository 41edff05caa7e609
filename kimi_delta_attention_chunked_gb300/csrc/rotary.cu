// rotary.cu -- rotary positions, and the append of latents with their rotated
// key part to the paged latent cache.
//
// A pair of channels (a, b) of a token at position p turns by the angle p f:
//     (a, b) -> factor (a cos p f - b sin p f,  b cos p f + a sin p f)
// with f the pair's frequency, in radians a position.  Pair i is (2 i, 2 i + 1) in the
// interleaved layout and (i, i + rot / 2) in the other.
//
// The angle.  In fp32, p f of a position of a million is off by up to 0.06.  What
// matters of it is its part of a turn, and that is exact in integers: F = f / (2 pi)
// as a 64-bit fraction of a turn (f has 24 bits, 1 / (2 pi) enters with 128), then p F
// modulo 2^64 is the angle, off by less than p 2^-64 turns.  The nearest quarter turn
// is taken off in integers too, and the rest, at most an eighth of a turn, is converted
// from all its 64 bits: with a relative error of 2^-24, however small it is.  sincospif
// gets an argument it has no reduction to do for.
#include <algorithm>

#include "latent.cuh"

namespace {

using kda_latent::kLatent;
using kda_latent::kRope;
using kda_latent::kRow;

// f / (2 pi) modulo 1, in units of 2^-64 turns
__device__ __forceinline__ uint64_t turns(float f) {
    constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;      // 2^128 / (2 pi)
    const uint32_t bits = __float_as_uint(f);
    const int e = (bits >> 23) & 0xff;
    const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);                     // f = m 2^(max(e, 1) - 150)
    const int shift = 150 - max(e, 1);
    const uint64_t lo = m * kHi, c = __umul64hi(m, kLo);
    const uint64_t sum = lo + c, top = __umul64hi(m, kHi) + (sum < lo ? 1 : 0);       // m / (2 pi) 2^64 = top : sum
    uint64_t t;
    if (shift >= 128) t = 0;
    else if (shift >= 64) t = top >> (shift - 64);
    else if (shift > 0) t = (sum >> shift) | (top << (64 - shift));
    else t = shift > -64 ? sum << -shift : 0;
    return bits >> 31 ? 0ull - t : t;
}

// (factor cos p f, factor sin p f)
__device__ __forceinline__ float2 turned(float f, int p, float factor) {
    if ((__float_as_uint(f) & 0x7f800000u) == 0x7f800000u) return make_float2(NAN, NAN);
    const uint64_t phase = turns(f) * (uint64_t)(int64_t)p;
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));                // [-2^61, 2^61)
    float s, c;
    sincospif((float)rest * 0x1p-63f, &s, &c);                                        // in half turns
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;                     // cos, sin up to their signs
    return make_float2(factor * ((quarter + 1) & 2 ? -x : x), factor * (quarter & 2 ? -y : y));
}

template <typename T>
__device__ __forceinline__ void turn(T& a, T& b, float2 cs) {
    const float x = kda::io<T>::ld(&a), y = kda::io<T>::ld(&b);
    kda::io<T>::st(&a, fmaf(x, cs.x, -y * cs.y));
    kda::io<T>::st(&b, fmaf(y, cs.x, x * cs.y));
}

constexpr int kThreads = 256;

struct RotarySizes {
    long long xt, xh, ot, oh;                          // strides in elements
    int T, H, d, rot, tokens;                          // tokens of a block
    int turned_items, copy_items, items;               // threads of a row: turned pieces, then copied ones
};

// A block takes `tokens` tokens: the cosines and sines of all their pairs once, into shared
// memory, then the rows (token, head).  A thread goes through them with one piece of the head's channels: VEC
// neighbouring channels of an interleaved head, VEC and their VEC partners of the other layout, or up to twice VEC
// channels that are copied (with one piece of those to a thread, 20,001 tokens x 32 heads of 128, half of
// them turned, took 75 us instead of 58).  The first row is fetched ahead of the table.  Bound: HBM for long prompts
// (0.83 of the copy rate there; two or four heads a thread 59 and 87 us: fewer threads fit; blocks of 16 and 32
// tokens 59 and 63 us), the launch and two dependent reads for decode steps (2.2 us).
template <typename T, int VEC, bool WIDE, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
kda_rotary_kernel(const T* x, const int32_t* __restrict__ positions, const float* __restrict__ inv_freq, RotarySizes s,
                  float factor, T* out) {
    extern __shared__ __align__(16) float2 table[];    // [tokens][rot / 2]
    kda_paged::wait_for_stream();
    const int half = s.rot >> 1, tid = threadIdx.x;
    const int t0 = blockIdx.x * s.tokens, n = min(s.tokens, s.T - t0);
    struct alignas(WIDE ? VEC * sizeof(T) : sizeof(T)) Piece { T v[VEC]; };
    const int per = kThreads / s.items, item = tid % s.items;             // rows at once
    const bool turns = item < s.turned_items;
    // first channels of the two pieces; the second may not be there
    const int c = turns ? item * VEC : s.rot + (item - s.turned_items) * VEC;
    const int c2 = turns ? half + c : c + s.copy_items * VEC;
    const bool two = turns ? !INTERLEAVED : c2 < s.d;
    const int len = WIDE ? VEC : min(VEC, s.d - c), len2 = WIDE ? VEC : min(VEC, s.d - c2);      // shorter at an odd end
    Piece p, q;
    auto load_piece = [&](Piece& y, const T* src, int m) {
        if (m == VEC) y = *reinterpret_cast<const Piece*>(src);
        else
            for (int i = 0; i < m; ++i) y.v[i] = src[i];
    };
    auto store_piece = [&](T* dst, const Piece& y, int m) {
        if (m == VEC) *reinterpret_cast<Piece*>(dst) = y;
        else
            for (int i = 0; i < m; ++i) dst[i] = y.v[i];
    };
    const int rows = n * s.H;
    auto load = [&](int row) {
        const int t = row / s.H, h = row - t * s.H;
        const T* src = x + (t0 + t) * s.xt + h * s.xh;
        load_piece(p, src + c, len);
        if (two) load_piece(q, src + c2, len2);
    };
    int row = tid / s.items < per ? tid / s.items : rows;
    if (row < rows) load(row);
    for (int e = tid; e < n * half; e += kThreads) {
        const int k = e / half;
        table[e] = turned(inv_freq[e - k * half], positions[t0 + k], factor);
    }
    __syncthreads();
    for (; row < rows; row += per) {
        const int t = row / s.H, h = row - t * s.H;
        T* dst = out + (t0 + t) * s.ot + h * s.oh;
        if (turns) {
            const float2* cs = table + t * half + (INTERLEAVED ? c >> 1 : c);
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) turn(p.v[i], p.v[i + 1], cs[i >> 1]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) turn(p.v[i], q.v[i], cs[i]);
            }
        }
        store_piece(dst + c, p, len);
        if (two) store_piece(dst + c2, q, len2);
        if (row + per < rows) load(row + per);
    }
}

template <typename T, int VEC, bool WIDE, bool INTERLEAVED>
cudaError_t rotary(const kda_host::RotaryArgs& a) {
    RotarySizes s{a.x_token, a.x_head, a.out_token, a.out_head, a.T, a.H, a.d, a.rot, 1, 0, 0, 0};
    s.turned_items = (INTERLEAVED ? a.rot : a.rot / 2) / VEC;
    const bool in_place = a.x == a.out;                // with the same strides: the other channels stay
    const int copied = in_place ? 0 : (a.d - a.rot + VEC - 1) / VEC;
    s.copy_items = (copied + 1) / 2;
    s.items = s.turned_items + s.copy_items;
    // a block's tokens share the set-up, and their rows hide each other's loads, as long as every SM
    // has a few blocks
    const int sms = kda_host::sm_count();
    while (s.tokens < 8 && a.T / (2 * s.tokens) >= 16 * sms) s.tokens *= 2;
    const int grid = (a.T + s.tokens - 1) / s.tokens;
    return kda_host::launch_overlapped(kda_rotary_kernel<T, VEC, WIDE, INTERLEAVED>, grid, kThreads,
                                       (size_t)s.tokens * (a.rot / 2) * sizeof(float2), a.stream, 1,
                                       static_cast<const T*>(a.x), a.positions, a.inv_freq, s, a.factor,
                                       static_cast<T*>(a.out));
}

template <typename T>
cudaError_t rotary_of(const kda_host::RotaryArgs& a) {
    constexpr int VEC = 16 / sizeof(T);
    auto aligned = [&](int64_t stride) { return stride % VEC == 0; };
    // 16-byte pieces where every piece of both tensors starts on a 16-byte boundary
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                      aligned(a.x_token) && aligned(a.x_head) && aligned(a.out_token) && aligned(a.out_head) &&
                      a.d % VEC == 0 && (a.interleaved ? a.rot : a.rot / 2) % VEC == 0;
    if (a.interleaved) return wide ? rotary<T, VEC, true, true>(a) : rotary<T, 2, false, true>(a);
    return wide ? rotary<T, VEC, true, false>(a) : rotary<T, 1, false, false>(a);
}

// One warp a token: 512 latent channels in 16-byte pieces (or one by one), and of the key part one
// pair a lane, which forms its own cosine and sine.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads)
kda_latent_append_kernel(const T* __restrict__ c, const T* __restrict__ k_rope, const int64_t* __restrict__ slot_map,
                         const int32_t* __restrict__ positions, const float* __restrict__ inv_freq, long long c_stride,
                         long long r_stride, int n_tokens, long long n_slots, int interleaved, float factor,
                         T* __restrict__ cache) {
    constexpr int VEC = 16 / sizeof(T);
    kda_paged::wait_for_stream();
    const int lane = threadIdx.x & 31;
    const int a = interleaved ? 2 * lane : lane, b = interleaved ? a + 1 : lane + kRope / 2;
    const float f = inv_freq ? inv_freq[lane] : 0.f;
    const int step = gridDim.x * (kThreads / 32);
    for (int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < n_tokens; t += step) {
        const long long slot = slot_map[t];
        const int pos = inv_freq ? positions[t] : 0;
        const T* src = c + t * c_stride;
        const T* rope = k_rope + t * r_stride;
        T* dst = cache + slot * kRow;
        T x = rope[a], y = rope[b];
        struct alignas(WIDE ? 16 : sizeof(T)) Piece { T v[WIDE ? VEC : 1]; };
        constexpr int N = kLatent / 32 / (WIDE ? VEC : 1);
        Piece p[N];
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = reinterpret_cast<const Piece*>(src)[lane + 32 * i];
        if (slot < 0 || slot >= n_slots) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<Piece*>(dst)[lane + 32 * i] = p[i];
        if (inv_freq) turn(x, y, turned(f, pos, factor));
        dst[kLatent + a] = x;
        dst[kLatent + b] = y;
    }
}

template <typename T>
cudaError_t latent_append(const kda_host::LatentAppendArgs& a) {
    const bool wide = reinterpret_cast<uintptr_t>(a.c) % 16 == 0 && a.c_stride * sizeof(T) % 16 == 0;
    const int grid = std::min((a.T + kThreads / 32 - 1) / (kThreads / 32), kda_host::sm_count() * 8);
    return kda_host::launch_overlapped(wide ? kda_latent_append_kernel<T, true> : kda_latent_append_kernel<T, false>, grid,
                                       kThreads, 0, a.stream, 1, static_cast<const T*>(a.c),
                                       static_cast<const T*>(a.k_rope), a.slot_map, a.positions, a.inv_freq, a.c_stride,
                                       a.r_stride, a.T, (long long)a.n_pages * a.page_size, a.interleaved, a.factor,
                                       static_cast<T*>(a.cache));
}

}  // namespace

namespace kda_host {

cudaError_t launch_rotary(const RotaryArgs& a) {
    return a.dtype == KDA_BF16 ? rotary_of<__nv_bfloat16>(a) : rotary_of<float>(a);
}

cudaError_t launch_latent_append(const LatentAppendArgs& a) {
    return a.dtype == KDA_BF16 ? latent_append<__nv_bfloat16>(a) : latent_append<float>(a);
}

}  // namespace kda_host
