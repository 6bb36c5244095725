// Decoding behind a shared prefix (minikv_decode_attn_prefix): the attention of
// every sharing sequence's query rows over one 2-bit prefix, read and
// dequantized once for up to 128 rows.  The partial softmax states are merged
// into each sequence's own step by the decode kernel (decode.cu).
//
// Both products are turned over, so that a tile of 128 tokens fills the M = 128
// of a tcgen05.mma and the N query rows (16, 32, 64 or 128) are its N:
//   S^T [128 tokens x N] = K^ [tokens x channels] Q^T,
//   O^T [128 channels x N] += V^^T [channels x tokens] P^T.
// With the rows as M a batch of 16 rows would pay for 128.
//
//   K^  fp16, the A operand in tensor memory: the thread of a token dequantizes
//       its 128 channels (rounded to fp16, the type the key was stored in before
//       it was quantized) and stores them to its own lane.
//   V^  fp16 in shared memory, [token][channel], read as an M-major A operand.
//   Q   [row][channel], P^T [token][row] in shared memory, the B operands.
// A code word's pairs (i, i + 8) come out of one mask each, so channels are
// kept in that order: position 16 w + 2 i + b is channel 16 w + i + 8 b.  Q is
// laid out alike, and the epilogue puts O^T's lanes back.
//
// Dequantization: c | 0x6400 is the fp16 number 1024 + c (code bits at mantissa
// bit 2I: 1024 + 4^I c), one fma makes it c exactly, a second c * scale + zero
// with one rounding.
//
// 20 warps: 1 issues the MMAs, 4-7 dequantize K, 8-11 V (a thread a token),
// 12-19 softmax (thread = token lane, half of the N columns each).  S, K^, V^
// and P have two buffers.  The reference max of a row moves only when a score
// passes it by 2^8; then the eight warps' column maxima meet in shared memory
// and O^T is rescaled.  Sums stay in registers, one a token lane and row, until
// the segment ends.
#include <math.h>

#include <mutex>

#include "common.cuh"
#include "prefix.cuh"
#include "tc.cuh"

namespace minikv {

namespace {

constexpr int kTile = 128;      // tokens of a tile
constexpr int kThreads = 640;
constexpr float kLazy = 8.f;
constexpr float kNone = -1e30f;

template <int N>
struct Smem {
    static constexpr int kNB = (N + 63) / 64;
    uint16_t v[2][2][kTile * 64];       // [stage][64-channel block][token][64], 128-byte swizzle
    uint16_t p[2][kNB][kTile * 64];     // [stage][64-row block][token][64]
    uint16_t q[2][N * 64];              // [64-channel block][row][64]
    uint32_t ksz[4][2][128];            // per K warp: scale pairs [64], zero pairs [64] of its group, two tiles
    float m[N], alpha[N];
    float wmax[4][N], wsum[4][N];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_done[2], drain;
    uint32_t tmem_base;
    int abort;
};

struct Args {
    PreTab tab;
    const uint32_t *k_codes, *v_codes;
    const uint16_t *k_scale, *k_zero, *v_scale, *v_zero, *k_res, *v_res;
    const uint16_t *q;
    float *part;
    unsigned *status;
    int Hq, Hkv, g, cap, G, lg2G, ring, n_packed, n_res, res_start;
    int rows, nt_packed;     // query rows of a KV head; token tiles of the packed part
    float scale_log2;
    short seq[MINIKV_MAX_RAGGED_SEQS];   // listed: sequence of each place
};

#ifndef MINIKV_WAIT_LIMIT
#define MINIKV_WAIT_LIMIT (1u << 26)
#endif

template <class S>
__device__ __forceinline__ bool wait(S &s, uint64_t *bar, uint32_t parity) {
    if (*reinterpret_cast<volatile int *>(&s.abort)) return false;
    if (mbar_wait(bar, parity, MINIKV_WAIT_LIMIT)) return true;
    *reinterpret_cast<volatile int *>(&s.abort) = 1;
    return false;
}
template <class S>
__device__ __forceinline__ bool wait_warp(S &s, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(s, bar, parity));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// fp16x2 (x, x) bits of 4^-I and -1024 * 4^-I
__host__ __device__ constexpr uint32_t pow_m(int I) { return 0x00010001u * (uint32_t)((15 - 2 * I) << 10); }
__host__ __device__ constexpr uint32_t neg_1024(int I) { return 0x00010001u * (0x8000u | (uint32_t)((25 - 2 * I) << 10)); }
// codes (i, i + 8) of a word as fp16x2; x = word, y = word >> 10
template <int I>
__device__ __forceinline__ uint32_t code2(uint32_t x, uint32_t y) {
    constexpr int J = I < 5 ? I : I - 5;
    const uint32_t t = ((I < 5 ? x : y) & (0x00030003u << (2 * J))) | 0x64006400u;
    return hfma2(t, pow_m(J), neg_1024(J));
}
// word `x` of 16 codes -> 8 fp16 pairs c * s + z; s and z as functions of the pair
template <class FS, class FZ>
__device__ __forceinline__ void dequant_word(uint32_t x, FS s, FZ z, uint32_t *out) {
    const uint32_t y = x >> 10;
    out[0] = hfma2(code2<0>(x, y), s(0), z(0));
    out[1] = hfma2(code2<1>(x, y), s(1), z(1));
    out[2] = hfma2(code2<2>(x, y), s(2), z(2));
    out[3] = hfma2(code2<3>(x, y), s(3), z(3));
    out[4] = hfma2(code2<4>(x, y), s(4), z(4));
    out[5] = hfma2(code2<5>(x, y), s(5), z(5));
    out[6] = hfma2(code2<6>(x, y), s(6), z(6));
    out[7] = hfma2(code2<7>(x, y), s(7), z(7));
}
// 16 fp16 channels (two 16-byte chunks) into pair order
__device__ __forceinline__ void pair_order(const uint4 &lo, const uint4 &hi, uint32_t *out) {
    const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        out[2 * i] = __byte_perm(a[i], b[i], 0x5410);
        out[2 * i + 1] = __byte_perm(a[i], b[i], 0x7632);
    }
}
__device__ __forceinline__ uint32_t or_over(int bar, uint32_t x) {   // over the 128 threads of a named barrier
    uint32_t y;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.or.pred p, %2, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(y) : "r"(x), "r"(bar) : "memory");
    return y;
}
__device__ __forceinline__ void sync_all() { asm volatile("barrier.cta.sync 0, %0;\n" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void sync_half(int bar) { asm volatile("barrier.cta.sync %0, 128;\n" ::"r"(bar) : "memory"); }
// largest of a warp's values (through the order of the bits as integers)
__device__ __forceinline__ float warp_max(float x) {
    int i = __float_as_int(x);
    i ^= (i >> 31) & 0x7fffffff;
    i = __reduce_max_sync(0xffffffffu, i);
    i ^= (i >> 31) & 0x7fffffff;
    return __int_as_float(i);
}

// One segment: CTA c's tiles of unit u.
struct Seg {
    int u, rt, kvh, x0, n;   // row tile, KV head, first token tile of the unit, tiles
};

// The segment's query rows (zero rows behind the last), and fresh references.
template <int N>
__device__ __forceinline__ void load_rows(Smem<N> &s, const Args &a, const Seg &sg, int tid) {
    for (int e = tid; e < N * 8; e += kThreads) {
        const int n = e >> 3, w = e & 7, row = sg.rt * N + n;
        uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (row < a.rows) {
            const int place = row / a.g, h = row - place * a.g;
            const int b = a.tab.listed ? a.seq[place] : place;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((size_t)b * a.Hq + sg.kvh * a.g + h) * kD) + 2 * w;
            pair_order(__ldg(src), __ldg(src + 1), out);
        }
        unsigned char *dst = reinterpret_cast<unsigned char *>(s.q[w >> 2]) + n * 128;
        const int ch = 2 * (w & 3);
        *reinterpret_cast<uint4 *>(dst + ((ch ^ (n & 7)) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4 *>(dst + (((ch + 1) ^ (n & 7)) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
    }
    if (tid < N) s.m[tid] = kNone;
    tc::fence_proxy_async_smem();
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ Args a) {
    constexpr int C = N / 2;                 // columns of a softmax thread
    constexpr int CH = C < 16 ? C : 16;      // columns in registers at a time
    constexpr uint32_t kColS = 0, kColO = 2 * N, kColK = 3 * N;
    constexpr uint32_t kCols = 3 * N + 128 <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    using S = Smem<N>;
    S &s = *reinterpret_cast<S *>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = warp & 3;
    const int c = blockIdx.x;

    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], 128);
            mbar_init(&s.k_empty[i], 1);
            mbar_init(&s.v_full[i], 128);
            mbar_init(&s.v_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 256);
            mbar_init(&s.o_done[i], 1);
        }
        mbar_init(&s.drain, 1);
        s.abort = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (warp == 1) tc::tmem_alloc(&s.tmem_base, kCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s.tmem_base;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;

    const int lo = (int)((long long)c * a.tab.T / a.tab.P), hi = (int)((long long)(c + 1) * a.tab.T / a.tab.P);
    int it = 0;   // tiles of the CTA before this segment: the barriers' phases run on

    // Every role runs the segments in step: the query rows, a block barrier, the
    // role's own work on the segment's tiles, a block barrier.  (Each role has its
    // own copy of this loop, behind its own register budget.)
    auto segments = [&](auto work) {
        for (int x = lo; x < hi;) {
            Seg sg;
            sg.u = x / a.tab.tpu;
            sg.rt = sg.u / a.Hkv;
            sg.kvh = sg.u - sg.rt * a.Hkv;
            sg.x0 = x - sg.u * a.tab.tpu;
            sg.n = min(hi, (sg.u + 1) * a.tab.tpu) - x;
            x += sg.n;
            load_rows<N>(s, a, sg, tid);
            sync_all();
            work(sg);
            it += sg.n;
            sync_all();   // the segment's barriers, Q, references and O^T are free
            tc::fence_after_sync();
            if (*reinterpret_cast<volatile int *>(&s.abort)) break;
        }
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
        segments([&](const Seg &sg) {
            // ---------------- MMA issuer
            if (warp == 1 && lane == 0) {
                constexpr uint32_t id_s = tc::idesc_f16(kTile, N, false, false);
                constexpr uint32_t id_o = tc::idesc_f16(kD, N, true, true);
                auto issue_s = [&](int k) {   // tile k of the CTA
                    const int st = k & 1;
                    if (!wait(s, &s.k_full[st], (k >> 1) & 1)) return false;
                    tc::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_ts(tmem + kColS + st * N, tmem + kColK + st * 64 + kk * 8,
                                   tc::sdesc_sw128(smem_addr(s.q[kk >> 2]) + (kk & 3) * 32, 16, 1024), id_s, kk > 0);
                    tc::commit(&s.s_full[st]);
                    tc::commit(&s.k_empty[st]);
                    return true;
                };
                bool ok = issue_s(it);
                for (int i = 0; ok && i < sg.n; ++i) {
                    const int k = it + i, st = k & 1;
                    if (i + 1 < sg.n && !(ok = issue_s(k + 1))) break;
                    ok = wait(s, &s.v_full[st], (k >> 1) & 1) && wait(s, &s.p_full[st], (k >> 1) & 1);
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_ss(tmem + kColO, tc::sdesc_sw128(smem_addr(s.v[st][0]) + kk * 2048, kTile * 128, 1024),
                                   tc::sdesc_sw128(smem_addr(s.p[st][0]) + kk * 2048, kTile * 128, 1024), id_o,
                                   (i > 0) || (kk > 0));
                    tc::commit(&s.o_done[st]);
                    tc::commit(&s.v_empty[st]);
                }
            }
            __syncwarp();
        });
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
        segments([&](const Seg &sg) {
            // ---------------- K: token 32 quad + lane of the tile
            const size_t plane = (size_t)sg.kvh;
            uint4 c0, c1;        // the token's codes
            uint2 ks, kz;        // four channels of the warp's group: scale, zero
            auto fetch = [&](int xt) {
                const int t = xt * kTile + 32 * quad;   // the warp's first token: all 32 in one group
                if (xt < a.nt_packed && t < a.n_packed) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.k_codes + (plane * a.cap + t + lane) * 8);
                    c0 = __ldg(src);
                    c1 = __ldg(src + 1);
                    const size_t grow = (plane * (a.cap >> a.lg2G) + (t >> a.lg2G)) * kD;
                    ks = __ldg(reinterpret_cast<const uint2 *>(a.k_scale + grow) + lane);
                    kz = __ldg(reinterpret_cast<const uint2 *>(a.k_zero + grow) + lane);
                }
            };
            fetch(sg.x0);
            for (int i = 0; i < sg.n; ++i) {
                const int k = it + i, st = k & 1, xt = sg.x0 + i;
                const bool packed = xt < a.nt_packed;
                uint32_t *sz = s.ksz[quad][st];
                const int t = (packed ? xt : xt - a.nt_packed) * kTile + 32 * quad;
                uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                if (packed) {
                    // lanes of channels 16w + 0..7 pair the scales, those of 16w + 8..15 the zeros
                    const bool up = lane & 2;
                    const uint2 mine = up ? kz : ks, give = up ? ks : kz;
                    uint2 got;
                    got.x = __shfl_xor_sync(0xffffffffu, give.x, 2);
                    got.y = __shfl_xor_sync(0xffffffffu, give.y, 2);
                    const uint2 a0 = up ? got : mine, b0 = up ? mine : got;
                    *reinterpret_cast<uint4 *>(sz + (up ? 64 : 0) + 8 * (lane >> 2) + 4 * (lane & 1)) =
                        make_uint4(__byte_perm(a0.x, b0.x, 0x5410), __byte_perm(a0.x, b0.x, 0x7632),
                                   __byte_perm(a0.y, b0.y, 0x5410), __byte_perm(a0.y, b0.y, 0x7632));
                    __syncwarp();
                }
                fetch(xt + 1);
                if (k >= 2 && !wait_warp(s, &s.k_empty[st], ((k >> 1) - 1) & 1)) break;
                tc::fence_after_sync();
                const uint32_t dst = tmem + lanes + kColK + st * 64;
                if (packed) {
                    const bool live = t < a.n_packed;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t out[32];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int wi = 4 * half + j;
                            const uint4 s0 = *reinterpret_cast<const uint4 *>(sz + 8 * wi);
                            const uint4 s1 = *reinterpret_cast<const uint4 *>(sz + 8 * wi + 4);
                            const uint4 z0 = *reinterpret_cast<const uint4 *>(sz + 64 + 8 * wi);
                            const uint4 z1 = *reinterpret_cast<const uint4 *>(sz + 64 + 8 * wi + 4);
                            const uint32_t sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
                            const uint32_t zv[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
                            dequant_word(w[wi], [&](int i2) { return sv[i2]; }, [&](int i2) { return zv[i2]; }, out + 8 * j);
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) out[j] = live ? out[j] : 0u;
                        tc::tmem_st32(dst + 32 * half, out);
                    }
                } else {
                    const int i0 = t + lane;
                    int slot = a.res_start + i0;
                    if (slot >= a.ring) slot -= a.ring;
                    const uint4 *src =
                        reinterpret_cast<const uint4 *>(a.k_res + (plane * a.ring + (i0 < a.n_res ? slot : 0)) * kD);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t out[32];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            pair_order(__ldg(src + 8 * half + 2 * j), __ldg(src + 8 * half + 2 * j + 1), out + 8 * j);
#pragma unroll
                        for (int j = 0; j < 32; ++j) out[j] = i0 < a.n_res ? out[j] : 0u;
                        tc::tmem_st32(dst + 32 * half, out);
                    }
                }
                tc::wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(&s.k_full[st]);
            }
        });
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
        segments([&](const Seg &sg) {
            // ---------------- V: token 32 quad + lane of the tile
            const size_t plane = (size_t)sg.kvh;
            const int r = 32 * quad + lane;
            uint4 c0, c1;
            uint32_t vs = 0, vz = 0;
            auto fetch = [&](int xt) {
                const int t = xt * kTile + r;
                if (xt < a.nt_packed && t < a.n_packed) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.v_codes + (plane * a.cap + t) * 8);
                    c0 = __ldg(src);
                    c1 = __ldg(src + 1);
                    vs = __ldg(a.v_scale + plane * a.cap + t);
                    vz = __ldg(a.v_zero + plane * a.cap + t);
                }
            };
            fetch(sg.x0);
            for (int i = 0; i < sg.n; ++i) {
                const int k = it + i, st = k & 1, xt = sg.x0 + i;
                const bool packed = xt < a.nt_packed;
                const int t = (packed ? xt : xt - a.nt_packed) * kTile + r;
                const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                const uint32_t s2 = vs * 0x00010001u, z2 = vz * 0x00010001u;
                fetch(xt + 1);
                if (k >= 2 && !wait_warp(s, &s.v_empty[st], ((k >> 1) - 1) & 1)) break;
                const bool live = t < (packed ? a.n_packed : a.n_res);
                int slot = a.res_start + t;
                if (slot >= a.ring) slot -= a.ring;
                const uint4 *src =
                    reinterpret_cast<const uint4 *>(a.v_res + (plane * a.ring + (!packed && live ? slot : 0)) * kD);
#pragma unroll
                for (int wi = 0; wi < 8; ++wi) {
                    uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};   // a token that is not there: P = 0 must not meet garbage
                    if (live) {
                        if (packed) dequant_word(w[wi], [&](int) { return s2; }, [&](int) { return z2; }, out);
                        else pair_order(__ldg(src + 2 * wi), __ldg(src + 2 * wi + 1), out);
                    }
                    unsigned char *dst = reinterpret_cast<unsigned char *>(s.v[st][wi >> 2]) + r * 128;
                    const int ch = 2 * (wi & 3);
                    *reinterpret_cast<uint4 *>(dst + ((ch ^ (r & 7)) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
                    *reinterpret_cast<uint4 *>(dst + (((ch + 1) ^ (r & 7)) << 4)) =
                        make_uint4(out[4], out[5], out[6], out[7]);
                }
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(&s.v_full[st]);
            }
        });
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;\n");
        segments([&](const Seg &sg) {
            // ---------------- softmax: token lane r, columns n0 .. n0 + C - 1
            const int half = warp >= 16, n0 = half * C, r = 32 * quad + lane, bar = 1 + half;
            const int rank = r;   // of the 128 threads of the half
            const float sc = a.scale_log2;
            float l[C];
#pragma unroll
            for (int j = 0; j < C; ++j) l[j] = 0.f;
            bool ok = true;
            for (int i = 0; i < sg.n; ++i) {
                const int k = it + i, st = k & 1, xt = sg.x0 + i;
                const bool live = xt < a.nt_packed ? xt * kTile + r < a.n_packed
                                                   : (xt - a.nt_packed) * kTile + r < a.n_res;
                ok = ok && wait_warp(s, &s.s_full[st], (k >> 1) & 1);
                tc::fence_after_sync();
                const uint32_t ts = tmem + lanes + kColS + st * N + n0;
                // does any score pass its row's reference by kLazy?
                float mx = -INFINITY;
#pragma unroll
                for (int j0 = 0; j0 < C; j0 += CH) {
                    uint32_t xr[CH];
                    tc::tmem_ld<CH>(ts + j0, xr);
                    tc::wait_ld();
#pragma unroll
                    for (int j = 0; j < CH; j += 4) {
                        const float4 m4 = *reinterpret_cast<const float4 *>(&s.m[n0 + j0 + j]);
                        mx = fmaxf(mx, fmaxf(fmaf(__uint_as_float(xr[j]), sc, -m4.x), fmaf(__uint_as_float(xr[j + 1]), sc, -m4.y)));
                        mx = fmaxf(mx, fmaxf(fmaf(__uint_as_float(xr[j + 2]), sc, -m4.z), fmaf(__uint_as_float(xr[j + 3]), sc, -m4.w)));
                    }
                }
                // (a failed wait joins the vote: the warps of a half leave the loop together, at this barrier)
                if (or_over(bar, !ok || (live && mx > kLazy))) {
                    if (or_over(bar, !ok)) {
                        ok = false;
                        break;
                    }
                    // column maxima of the tile -> new references; sums and O^T follow
#pragma unroll 1
                    for (int j = 0; j < C; j += 8) {
                        uint32_t xr[8];
                        tc::tmem_ld<8>(ts + j, xr);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float top = warp_max(live ? __uint_as_float(xr[e]) : -INFINITY);
                            if (lane == 0) s.wmax[quad][n0 + j + e] = top;
                        }
                    }
                    sync_half(bar);
                    if (rank < C) {
                        const int n = n0 + rank;
                        const float top = fmaxf(fmaxf(s.wmax[0][n], s.wmax[1][n]), fmaxf(s.wmax[2][n], s.wmax[3][n])) * sc;
                        const float old = s.m[n], now = fmaxf(old, top);
                        s.m[n] = now;
                        s.alpha[n] = ex2(old - now);
                    }
                    sync_half(bar);
#pragma unroll
                    for (int j = 0; j < C; ++j) l[j] *= s.alpha[n0 + j];
                    if (i > 0) {
                        ok = wait_warp(s, &s.o_done[(k - 1) & 1], ((k - 1) >> 1) & 1);
                        tc::fence_after_sync();
                        const uint32_t to = tmem + lanes + kColO + n0;
#pragma unroll 1
                        for (int j = 0; ok && j < C; j += 8) {
                            uint32_t o[8];
                            tc::tmem_ld<8>(to + j, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * s.alpha[n0 + j + e]);
                            tc::tmem_st<8>(to + j, o);
                        }
                        tc::wait_st();
                    }
                }
                // P of two tiles ago has been read
                if (k >= 2) ok = ok && wait_warp(s, &s.o_done[st], ((k >> 1) - 1) & 1);
                if (!ok) continue;   // to the next tile's vote, or the epilogue
#pragma unroll
                for (int j0 = 0; j0 < C; j0 += CH) {
                    uint32_t xr[CH];
                    tc::tmem_ld<CH>(ts + j0, xr);
                    tc::wait_ld();
#pragma unroll
                    for (int j = 0; j < CH; j += 8) {
                        uint32_t ph[4];
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            const float4 m4 = *reinterpret_cast<const float4 *>(&s.m[n0 + j0 + j + e]);
                            const float p0 = live ? ex2(fmaf(__uint_as_float(xr[j + e]), sc, -m4.x)) : 0.f;
                            const float p1 = live ? ex2(fmaf(__uint_as_float(xr[j + e + 1]), sc, -m4.y)) : 0.f;
                            const float p2 = live ? ex2(fmaf(__uint_as_float(xr[j + e + 2]), sc, -m4.z)) : 0.f;
                            const float p3 = live ? ex2(fmaf(__uint_as_float(xr[j + e + 3]), sc, -m4.w)) : 0.f;
                            l[j0 + j + e] += p0;
                            l[j0 + j + e + 1] += p1;
                            l[j0 + j + e + 2] += p2;
                            l[j0 + j + e + 3] += p3;
                            ph[e / 2] = pack_half2(p0, p1);
                            ph[e / 2 + 1] = pack_half2(p2, p3);
                        }
                        const int n = n0 + j0 + j, blkn = n >> 6, ch = (n & 63) >> 3;
                        *reinterpret_cast<uint4 *>(reinterpret_cast<unsigned char *>(s.p[st][blkn]) + r * 128 +
                                                   ((ch ^ (r & 7)) << 4)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                    }
                }
                tc::fence_proxy_async_smem();
                tc::fence_before_sync();
                tc::mbar_arrive(&s.p_full[st]);
            }
            // ---------------- epilogue: the segment's state to slot c + u
            const int last = it + sg.n - 1;
            if (ok) ok = wait_warp(s, &s.o_done[last & 1], (last >> 1) & 1);
            // sums over the 32 lanes: column j of a block of CH ends in lanes j (mod CH)
#pragma unroll
            for (int j0 = 0; j0 < C; j0 += CH) {
#pragma unroll
                for (int w = CH / 2; w >= 1; w >>= 1) {
                    const bool up = lane & w;
#pragma unroll
                    for (int j = 0; j < w; ++j) {
                        const float keep = up ? l[j0 + j + w] : l[j0 + j], give = up ? l[j0 + j] : l[j0 + j + w];
                        l[j0 + j] = keep + __shfl_xor_sync(0xffffffffu, give, w);
                    }
                }
                float t = l[j0];
#pragma unroll
                for (int w = CH; w < 32; w <<= 1) t += __shfl_xor_sync(0xffffffffu, t, w);
                if (lane < CH) s.wsum[quad][n0 + j0 + lane] = t;
            }
            sync_half(bar);
            if (ok) {
                tc::fence_after_sync();
                float *base = a.part + (size_t)(c + sg.u) * N * kPreStride;
                const int pos = r & 15, ch = (r & ~15) + (pos >> 1) + 8 * (pos & 1);
                const uint32_t to = tmem + lanes + kColO + n0;
                const int rows = min(C, a.rows - sg.rt * N - n0);   // rows behind the last are not written
#pragma unroll 1
                for (int j = 0; j < C; j += 8) {
                    uint32_t o[8];
                    tc::tmem_ld<8>(to + j, o);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (j + e < rows) base[(size_t)(n0 + j + e) * kPreStride + ch] = __uint_as_float(o[e]);
                }
                if (rank < rows) {
                    const int n = n0 + rank;
                    base[(size_t)n * kPreStride + 128] = s.m[n];
                    base[(size_t)n * kPreStride + 129] = s.wsum[0][n] + s.wsum[1][n] + s.wsum[2][n] + s.wsum[3][n];
                }
            }
            tc::fence_before_sync();
        });
    }
    if (warp == 1) {
        if (lane == 0) {   // every MMA issued has finished (after an expired wait, too)
            tc::commit(&s.drain);
            mbar_wait(&s.drain, 0);
        }
        __syncwarp();
        tc::tmem_dealloc(tmem, kCols);
    }
    if (tid == 0) a.status[c] = s.abort ? 1u : 0u;
}

std::mutex g_mu;
bool g_attr[kMaxDevices] = {};
int g_sms[kMaxDevices] = {};

constexpr int kMaxCtas = 148;   // one a SM

int row_tile(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

template <int N>
int launch(const Args &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.tab.P);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem<N>) + 1024;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, prefix_kernel<N>, a);
    return check_launch("decode_attn_prefix: prefix pass");
}

template <int N>
bool set_attr() {
    return cudaFuncSetAttribute(prefix_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Smem<N>) + 1024) == cudaSuccess;
}

}  // namespace

// Workspace of the prefix pass: a status word a CTA, then the partial states.
size_t prefix_status_words() { return kMaxCtas; }
static size_t prefix_status_bytes() { return (kMaxCtas * 4 + 255) / 256 * 256; }
size_t prefix_workspace_bytes(int B, int Hq, int Hkv) {
    const long long rows = (long long)B * (Hq / Hkv);
    const int N = row_tile(rows);
    const size_t units = (size_t)((rows + N - 1) / N) * Hkv;
    return prefix_status_bytes() + (kMaxCtas + units) * N * kPreStride * 4;
}

// Queue the prefix pass: states of the sharing sequences' rows over `p`, and *tab for the merging decode kernel.
// ws: prefix_workspace_bytes.  shared: host flags a sequence, or NULL (all).  tab->P = 0: nobody attends to anything.
int prefix_launch(const minikv_cache *p, const int *shared, int B, const uint16_t *q, int Hq, float sm_scale, void *ws,
                  cudaStream_t stream, PreTab *tab) {
    Args a;
    PreTab &t = a.tab;
    const int Hkv = p->Hkv, g = Hq / Hkv;
    int places = B;
    t.listed = 0;
    if (shared) {
        t.listed = 1;
        places = 0;
        for (int b = 0; b < B; ++b) {
            t.place[b] = shared[b] ? (short)places : (short)-1;
            if (shared[b]) a.seq[places++] = (short)b;
        }
    }
    const int n_packed = p->seq ? p->seq[0] : p->n_packed, n_res = p->seq ? p->seq[1] : p->n_res;
    t.P = 0;
    t.part = reinterpret_cast<float *>(static_cast<char *>(ws) + prefix_status_bytes());
    a.status = static_cast<unsigned *>(ws);
    if (places == 0 || n_packed + n_res == 0) {
        *tab = t;
        if (cudaMemsetAsync(ws, 0, prefix_status_bytes(), stream) != cudaSuccess)
            return check_launch("decode_attn_prefix: clearing the status words");
        return MINIKV_OK;
    }
    a.rows = places * g;
    const int N = row_tile(a.rows);
    t.lgN = N == 16 ? 4 : N == 32 ? 5 : N == 64 ? 6 : 7;
    a.nt_packed = (n_packed + kTile - 1) / kTile;
    t.tpu = a.nt_packed + (n_res + kTile - 1) / kTile;
    const long long T = (long long)((a.rows + N - 1) / N) * Hkv * t.tpu;
    if (T > 0x7fffffff) return fail(MINIKV_ERR_UNSUPPORTED, "decode_attn_prefix: more than 2^31 tiles of work");
    t.T = (int)T;
    const int dev = current_device();
    if (dev < 0) return fail(MINIKV_ERR_CUDA, "decode_attn_prefix: no current CUDA device");
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!g_attr[dev]) {
            if (!set_attr<16>() || !set_attr<32>() || !set_attr<64>() || !set_attr<128>())
                return check_launch("decode_attn_prefix: attribute");
            int sms = kMaxCtas;
            if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) sms = kMaxCtas;
            g_sms[dev] = sms < kMaxCtas ? sms : kMaxCtas;
            g_attr[dev] = true;
        }
        t.P = g_sms[dev];
    }
    if (t.P > t.T) t.P = t.T;
    a.k_codes = p->k_codes; a.v_codes = p->v_codes;
    a.k_scale = p->k_scale; a.k_zero = p->k_zero; a.v_scale = p->v_scale; a.v_zero = p->v_zero;
    a.k_res = p->k_res; a.v_res = p->v_res;
    a.q = q;
    a.part = const_cast<float *>(t.part);
    a.Hq = Hq; a.Hkv = Hkv; a.g = g; a.cap = p->cap; a.G = p->G;
    a.lg2G = 31 - __builtin_clz((unsigned)p->G);
    a.ring = p->R + p->G;
    a.n_packed = n_packed;
    a.n_res = n_res;
    a.res_start = p->seq ? p->seq[2] : p->res_start;
    a.scale_log2 = sm_scale * kLog2e;
    *tab = t;
    switch (N) {
        case 16: return launch<16>(a, stream);
        case 32: return launch<32>(a, stream);
        case 64: return launch<64>(a, stream);
        default: return launch<128>(a, stream);
    }
}

}  // namespace minikv
