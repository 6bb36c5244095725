// Decoding behind a shared prefix (minikv_decode_attn_prefix): the attention of
// every sharing sequence's query rows over one 2-bit prefix, read and
// dequantized once for up to 128 rows.  The partial softmax states are merged
// into each sequence's own step by the decode kernel (decode.cu).
//
// Both products are turned over, so that a tile of 128 tokens fills the M = 128
// of a tcgen05.mma and the N query rows (16, 32, 64 or 128) are its N:
//   S'^T [128 tokens x N] = K' [tokens x channels] Q^T,
//   O'^T [128 channels x N] += V'^T [channels x tokens] P^T.
// With the rows as M a batch of 16 rows would pay for 128.
//
// Exact operands.  A dequantized c s + z needs more than fp16's 11 bits, but
// (c - o) s / 2 with o = 1 or 2 is a whole multiple of s / 2 between -2 and 2: an
// fp16 number, never above the largest.  (Where s is an odd multiple of fp16's
// smallest step, half of it is not: s / 2, and a residual token's halved channel,
// are then off by at most 2^-25.)  With c s + z = (c - o) s + (z + o s):
//   score = 2 K' q + T,  T = q (z + s), one number a (key group, row), o = 1;
//   out   = 2 V' p + sum_t p_t (z + o s)_t, one number a row; o = 1 for even, 2
//           for odd tokens, so that both sums stay near the output's size (the
//           tensor cores' long sums lose bits of the larger).
// Both corrections, and the sum of p, are small products on mma.sync with fp32
// sums: T = Q [z | s] of the tile's four 32-token quarters (each within one key
// group), and [1; hi(z + o s); lo(z + o s)] P.  Only P is rounded (to fp16, half
// a step of the output's own type).
//
//   K'  fp16, the A operand in tensor memory: the thread of a token dequantizes
//       its 128 channels and stores them to its own lane.
//   V'  fp16 in shared memory, [token][channel], read as an M-major A operand.
//   Q   [row][channel], P^T [token][row] in shared memory, the B operands.
// A code word's pairs (i, i + 8) come out of one mask each, so channels are
// kept in that order: position 16 w + 2 i + b is channel 16 w + i + 8 b.  Q is
// laid out alike, and the epilogue puts O'^T's lanes back.
//
// Dequantization: c | 0x6400 is the fp16 number 1024 + c (code bits at mantissa
// bit 2I: 1024 + 4^I c); one fma makes it (c - o) / 2, one product (c - o) s / 2.
//
// 32 warps: 0 and 2 compute T (half of the rows each), 1 and 3 issue the MMAs of
// the two products, 4-7 dequantize K, 8-11 V (a thread a token), 12-27 softmax
// (thread = token lane, a quarter of the rows each; N = 16: two halves, 20-27
// idle), 28-31 the sums over P (a quarter of the rows each).  S, K', V' and P
// have two buffers.  The reference max of a row moves only when a score passes it
// by 2^8; then the column maxima of a part's four warps meet in shared memory and
// O'^T and the sums are rescaled.
//
// What bounds it: the roles' chains of short dependent steps, at about 0.6
// instructions a cycle and SM quarter.  Under running MMAs a shared-memory load
// takes 200-400 cycles and a wait that is over 250, so the softmax warps wait
// once a tile and loads are asked for ahead (one wait instead of three: 461 -> 437
// us a step at 96 sequences x 131000 tokens; 16 softmax warps instead of 8, with
// every score in registers: 437 -> 402).  The loops are kept short on purpose:
// with the roles unrolled over their tiles, half of the warps waited for
// instructions (3.3 us a tile at N = 64, now 1.5).  The pass takes 21 us behind
// 4321 tokens (24 sequences, 32 KV heads, N = 32), 34 us behind 32768 (16
// sequences, N = 64) and 345 us behind 131000 (96 sequences, three tiles of 128
// rows: 600 TFLOP/s).
#include <math.h>

#include <mutex>

#include "common.cuh"
#include "prefix.cuh"
#include "tc.cuh"

namespace minikv {

namespace {

constexpr int kTile = 128;      // tokens of a tile
constexpr int kThreads = 1024;
constexpr int kMaxCtas = 148;   // one a SM
constexpr float kLazy = 8.f;
// words of a quarter's scales and zeros: the eight columns that T reads side by side lie in distinct banks
constexpr int kKszZero = 68, kKszStride = 136;

template <int N>
struct Smem {
    static constexpr int kNB = (N + 63) / 64;
    uint16_t v[2][2][kTile * 64];       // [stage][64-channel block][token][64], 128-byte swizzle
    uint16_t p[2][kNB][kTile * 64];     // [stage][64-row block][token][64]
    uint16_t q[2][N * 64];              // [64-channel block][row][64]
    uint32_t ksz[8][4][kKszStride];     // [tile & 7][quarter]: scale pairs [64], zero pairs [64] of its key group
    uint32_t vz[2][2][kTile / 2];       // [stage][hi, lo]: fp16 z + o s of the value tokens
    float tz[4][4][N];                  // [tile & 3][quarter][row]: T in log2 units
    float bias[16][N / 2];              // a softmax warp's T - reference of the tile in hand
    float m[N], alpha[2][N], l[N], pz[N];
    float wmax[4][N];
    int resc[2][4];                     // [stage][part]: the tile moved the references (alpha holds the factors)
    uint64_t k_full[2], k_empty[2], kz_full[8], v_full[2], s_full[2], p_full[2], o_done[2], drain[2];   // in this order
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

template <class S>
__device__ __forceinline__ bool wait_warp(S &s, uint64_t *bar, uint32_t parity) {
    return tc::role_wait_warp(&s.abort, bar, parity);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
constexpr uint32_t kHalf2 = 0x38003800u;   // fp16x2 (0.5, 0.5)
// fp16x2 bits of 4^-I / 2 and of -(1024 4^-I + o) / 2, o = 1 (512.5, 128.5, 32.5, 8.5, 2.5) or 2 (513, 129, 33, 9, 3)
__host__ __device__ constexpr uint32_t code_mul(int I) { return 0x00010001u * (uint32_t)((14 - 2 * I) << 10); }
__host__ __device__ constexpr uint32_t code_add(int I, int o) {
    return 0x00010001u * (0x8000u | (uint32_t)((24 - 2 * I) << 10) | ((uint32_t)o << (2 * I)));
}
// The offset of a lane's token, as the five addends above.
struct Offset {
    uint32_t add[5];
    __device__ __forceinline__ explicit Offset(bool two) {
#pragma unroll
        for (int i = 0; i < 5; ++i) add[i] = two ? code_add(i, 2) : code_add(i, 1);
    }
};
// (c - o) / 2 of codes (i, i + 8) of a word as fp16x2; x = word, y = word >> 10
template <int I>
__device__ __forceinline__ uint32_t code2(uint32_t x, uint32_t y, const Offset &o) {
    constexpr int J = I < 5 ? I : I - 5;
    const uint32_t t = ((I < 5 ? x : y) & (0x00030003u << (2 * J))) | 0x64006400u;
    return hfma2(t, code_mul(J), o.add[J]);
}
// word `x` of 16 codes -> 8 fp16 pairs (c - o) s / 2; s as a function of the pair
template <class FS>
__device__ __forceinline__ void dequant_word(uint32_t x, const Offset &o, FS s, uint32_t *out) {
    const uint32_t y = x >> 10;
    out[0] = hmul2(code2<0>(x, y, o), s(0));
    out[1] = hmul2(code2<1>(x, y, o), s(1));
    out[2] = hmul2(code2<2>(x, y, o), s(2));
    out[3] = hmul2(code2<3>(x, y, o), s(3));
    out[4] = hmul2(code2<4>(x, y, o), s(4));
    out[5] = hmul2(code2<5>(x, y, o), s(5));
    out[6] = hmul2(code2<6>(x, y, o), s(6));
    out[7] = hmul2(code2<7>(x, y, o), s(7));
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
// Column maxima of a warp's [32 lanes x C]: x[0] of lane l becomes that of column
// l / (32 / C).  Lanes a bit apart halve their columns between them, step by step.
template <int C, int BIT>
__device__ __forceinline__ void col_max(float *x, int lane) {
    if constexpr (BIT > 0) {
        if constexpr (C > 1) {
            const bool up = lane & BIT;
#pragma unroll
            for (int j = 0; j < C / 2; ++j) {
                const float keep = up ? x[j + C / 2] : x[j], give = up ? x[j] : x[j + C / 2];
                x[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, BIT));
            }
            col_max<C / 2, BIT / 2>(x, lane);
        } else {
            x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], BIT));
            col_max<1, BIT / 2>(x, lane);
        }
    }
}

// One segment: CTA c's tiles of unit u.
struct Seg {
    int u, rt, kvh, x0, n;   // row tile, KV head, first token tile of the unit, tiles
};

// The segment's query rows (zero rows behind the last), and fresh references; thread tid of T.
template <int N, int T>
__device__ __forceinline__ void load_rows(Smem<N> &s, const Args &a, const Seg &sg, int tid) {
#pragma unroll 1
    for (int e = tid; e < N * 8; e += T) {
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
    if (tid < N) s.m[tid] = 0.f;   // the first tile sets it to its maximum
    tc::fence_proxy_async_smem();
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ Args a) {
    constexpr int kP = N == 16 ? 2 : 4;      // softmax groups: parts of the rows
    constexpr int C = N / kP;                // rows of a softmax thread
    constexpr int kTW = N == 16 ? 1 : 2;     // T warps
    constexpr int kSW = N == 16 ? 2 : 4;     // sum warps
    constexpr uint32_t kColS = 0, kColO = 2 * N, kColK = 3 * N;
    constexpr uint32_t kCols = 3 * N + 128 <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    using S = Smem<N>;
    S &s = *reinterpret_cast<S *>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
    // (broadcast: the compiler then knows that branches on the warp, and descriptors behind them, are uniform)
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), quad = warp & 3;
    const int g_ = lane >> 2, t_ = lane & 3;
    const int c = blockIdx.x;

    if (warp == 0) {
        // arrivals a phase: k_full 4 (warps), k_empty S, kz_full 4 (eight barriers), v_full 4, s_full S and the T warps,
        // p_full the softmax warps, o_done O'^T and the sum warps, drain 1
        constexpr unsigned long long kCounts = 4ull | 1ull << 8 | 4ull << 16 | 4ull << 24 | (1ull + kTW) << 32 |
                                               (4ull * kP) << 40 | (1ull + kSW) << 48 | 1ull << 56;
        const int kind = lane < 4 ? lane >> 1 : lane < 12 ? 2 : (lane >> 1) - 3;
        if (lane < 22) mbar_init(&s.k_full[0] + lane, (uint32_t)(kCounts >> (8 * kind)) & 255u);
        fence_mbar_init();
        if (lane == 0) s.abort = 0;
    }
    // The dependents are let go only once everything before this kernel is done: the decode kernel of the step
    // then starts where SMs are free, with all of its inputs in place, and waits for this grid only where it
    // merges this grid's states.
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (warp == 1) tc::tmem_alloc(&s.tmem_base, kCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem_base, 0);
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;

    const int lo = (int)((long long)c * a.tab.T / a.tab.P), hi = (int)((long long)(c + 1) * a.tab.T / a.tab.P);
    int it = 0;   // tiles of the CTA before this segment: the barriers' phases run on
    // phase parity of tile k's use of a two-stage barrier, and of the use before it
    auto ph = [](int k) { return (uint32_t)(k >> 1) & 1; };
    auto ph_prev = [](int k) { return (uint32_t)((k >> 1) - 1) & 1; };

    // Every role runs the segments in step: what the role does before (the first
    // tile's loads, the query rows), a block barrier, the role's work on the
    // segment's tiles, a block barrier.  (Each role has its own copy of this loop,
    // behind its own register budget.)
    auto segments = [&](auto before, auto work) {
        for (int x = lo; x < hi;) {
            Seg sg;
            sg.u = x / a.tab.tpu;
            sg.rt = sg.u / a.Hkv;
            sg.kvh = sg.u - sg.rt * a.Hkv;
            sg.x0 = x - sg.u * a.tab.tpu;
            sg.n = min(hi, (sg.u + 1) * a.tab.tpu) - x;
            x += sg.n;
            before(sg);
            sync_all();
            work(sg);
            it += sg.n;
            sync_all();   // the segment's barriers, Q, references and O'^T are free
            tc::fence_after_sync();
            if (*reinterpret_cast<volatile int *>(&s.abort)) break;
        }
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 72;\n");
        segments([](const Seg &) {}, [&](const Seg &sg) {
            if (warp == 0 || (warp == 2 && kTW == 2)) {
                // ---------------- T [rows x quarters] = Q [z | s], 16-row tiles MT0 .. MT0 + MT - 1
                constexpr int MT = N / 16 / kTW;   // 16-row tiles of a warp
                const float sc = a.scale_log2;
                const int lrow = (lane & 7) + 8 * ((lane >> 3) & 1), lch = lane >> 4;
                const uint32_t qrow = smem_addr(s.q[0]) + ((warp >> 1) * MT * 16 + lrow) * 128;
                // a 16-row tile's Q, the next one's asked for behind the products (a load takes 400 cycles under MMAs)
                uint32_t qa[8][4];
                auto load_q = [&](int m) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        ldmatrix_x4(qa[kk], qrow + m * 2048 + (kk >> 2) * (N * 128) + (((2 * (kk & 3) + lch) ^ (lrow & 7)) << 4));
                };
                load_q(0);
                for (int i = 0; i < sg.n; ++i) {
                    const int k = it + i, st = k & 1;
                    const uint32_t keep = sg.x0 + i < a.nt_packed ? 0xffffffffu : 0u;   // fp16 tokens have no T
                    // (tz of four tiles ago has been read: the last tile's wait below was for P of three ago)
                    if (!wait_warp(s, &s.kz_full[k & 7], (uint32_t)(k >> 3) & 1)) break;
                    // column g_: z of quarter g_, then s of quarter g_ - 4
                    const uint32_t *col = s.ksz[k & 7][g_ & 3] + (g_ < 4 ? kKszZero : 0) + t_;
                    float *tz = &s.tz[k & 3][2 * (t_ & 1)][(warp >> 1) * MT * 16 + g_];
                    uint32_t bz[8][2];
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        bz[kk][0] = col[8 * kk] & keep;
                        bz[kk][1] = col[8 * kk + 4] & keep;
                    }
#pragma unroll 1
                    for (int m = 0; m < MT; ++m) {
                        float d[2][4];
#pragma unroll
                        for (int e = 0; e < 8; ++e) (&d[0][0])[e] = 0.f;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) mma16816(d[kk & 1], qa[kk], bz[kk][0], bz[kk][1]);
                        if (MT > 1) load_q(m + 1 < MT ? m + 1 : 0);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v = d[0][e] + d[1][e];
                            v += __shfl_xor_sync(0xffffffffu, v, 2);
                            if (t_ < 2) tz[(e & 1) * N + 16 * m + 8 * (e >> 1)] = v * sc;
                        }
                    }
                    // P and the factors of two tiles ago have been read (waited for here: the softmax warps then wait
                    // once a tile, and a wait that is over takes 250 cycles)
                    if (k >= 2 && !wait_warp(s, &s.o_done[st], ph_prev(k))) break;
                    tc::arrive_warp(&s.s_full[st]);
                }
            } else if (warp == 1) {
                // ---------------- S'^T = K' Q^T (the warp waits together, one lane issues)
                constexpr uint32_t id_s = tc::idesc_f16(kTile, N, false, false);
                const uint64_t qd = tc::sdesc_sw128(smem_addr(s.q[0]), 16, 1024);
                for (int i = 0; i < sg.n; ++i) {
                    const int k = it + i;
                    const uint32_t st = k & 1;
                    // S of two tiles ago has been read
                    if (!wait_warp(s, &s.k_full[st], ph(k)) || (k >= 2 && !wait_warp(s, &s.p_full[st], ph_prev(k)))) break;
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)   // descriptors count 16-byte units
                            tc::mma_ts(tmem + kColS + st * N, tmem + kColK + st * 64 + kk * 8,
                                       qd + (kk >> 2) * (N * 8) + (kk & 3) * 2, id_s, kk > 0);
                        tc::commit(&s.s_full[st]);
                        tc::commit(&s.k_empty[st]);
                    }
                    __syncwarp();
                }
            } else if (warp == 3) {
                // ---------------- O'^T += V'^T P^T
                constexpr uint32_t id_o = tc::idesc_f16(kD, N, true, true);
                const uint64_t vd = tc::sdesc_sw128(smem_addr(s.v[0][0]), kTile * 128, 1024);
                const uint64_t pd = tc::sdesc_sw128(smem_addr(s.p[0][0]), kTile * 128, 1024);
                for (int i = 0; i < sg.n; ++i) {
                    const int k = it + i;
                    const uint32_t st = k & 1;
                    if (!wait_warp(s, &s.v_full[st], ph(k)) || !wait_warp(s, &s.p_full[st], ph(k))) break;
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
                        const uint64_t v = vd + st * (2 * kTile * 8), p = pd + st * (S::kNB * kTile * 8);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            tc::mma_ss(tmem + kColO, v + kk * 128, p + kk * 128, id_o, (i > 0) || (kk > 0));
                        tc::commit(&s.o_done[st]);
                    }
                    __syncwarp();
                }
            }
        });
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        uint4 c0, c1;        // the token's codes
        uint2 ks, kz;        // four channels of the quarter's group: scale, zero
        auto fetch = [&](size_t plane, int xt) {
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
        segments([&](const Seg &sg) { fetch(sg.kvh, sg.x0); }, [&](const Seg &sg) {
            // ---------------- K: token 32 quad + lane of the tile
            const size_t plane = (size_t)sg.kvh;
            const Offset off(false);
            for (int i = 0; i < sg.n; ++i) {
                const int k = it + i, st = k & 1, xt = sg.x0 + i;
                const bool packed = xt < a.nt_packed;
                uint32_t *sz = s.ksz[k & 7][quad];
                const int t = (packed ? xt : xt - a.nt_packed) * kTile + 32 * quad;
                uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                // lanes of channels 16w + 0..7 pair the scales, those of 16w + 8..15 the zeros
                const bool up = lane & 2;
                const uint2 mine = up ? kz : ks, give = up ? ks : kz;
                uint2 got;
                got.x = __shfl_xor_sync(0xffffffffu, give.x, 2);
                got.y = __shfl_xor_sync(0xffffffffu, give.y, 2);
                const uint2 a0 = up ? got : mine, b0 = up ? mine : got;
                fetch(plane, xt + 1);
                // (T of eight tiles ago is done with its scales: the last tile's wait below was for S of three ago, S comes
                // after P of two tiles before it, and P after its tile's T: that is T of five ago)
                *reinterpret_cast<uint4 *>(sz + (up ? kKszZero : 0) + 8 * (lane >> 2) + 4 * (lane & 1)) =
                    make_uint4(__byte_perm(a0.x, b0.x, 0x5410), __byte_perm(a0.x, b0.x, 0x7632),
                               __byte_perm(a0.y, b0.y, 0x5410), __byte_perm(a0.y, b0.y, 0x7632));
                tc::arrive_warp(&s.kz_full[k & 7]);
                if (k >= 2 && !wait_warp(s, &s.k_empty[st], ph_prev(k))) break;
                tc::fence_after_sync();
                const uint32_t dst = tmem + lanes + kColK + st * 64;
                if (packed && t < a.n_packed) {
                    uint32_t d = dst;
                    const uint32_t *sp = sz;
                    // two words an iteration, each one's scales asked for a word ahead (behind the last word: the zeros)
                    uint4 sv[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) sv[j] = *reinterpret_cast<const uint4 *>(sp + 4 * j);
#pragma unroll 1
                    for (int wi = 0; wi < 4; ++wi, d += 16) {
                        sp += 16;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint4 s0 = sv[2 * j], s1 = sv[2 * j + 1];
                            const uint32_t pair[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
                            uint32_t out[8];
                            dequant_word(w[j], off, [&](int i2) { return pair[i2]; }, out);
                            tc::tmem_st<8>(d + 8 * j, out);
                            sv[2 * j] = *reinterpret_cast<const uint4 *>(sp + 8 * j);
                            sv[2 * j + 1] = *reinterpret_cast<const uint4 *>(sp + 8 * j + 4);
                        }
#pragma unroll
                        for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
                    }
                } else if (packed) {   // a quarter behind the last packed token
                    uint32_t out[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) out[e] = 0u;
#pragma unroll 1
                    for (int wi = 0; wi < 4; ++wi) tc::tmem_st<16>(dst + 16 * wi, out);
                } else {
                    const int i0 = t + lane;
                    int slot = a.res_start + i0;
                    if (slot >= a.ring) slot -= a.ring;
                    const uint4 *src =
                        reinterpret_cast<const uint4 *>(a.k_res + (plane * a.ring + (i0 < a.n_res ? slot : 0)) * kD);
#pragma unroll 1
                    for (int w0 = 0; w0 < 8; w0 += 2) {   // two words in flight
                        uint4 x[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = __ldg(src + 2 * w0 + j);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t out[8];
                            pair_order(x[2 * j], x[2 * j + 1], out);
#pragma unroll
                            for (int e = 0; e < 8; ++e) out[e] = i0 < a.n_res ? hmul2(out[e], kHalf2) : 0u;
                            tc::tmem_st<8>(dst + 8 * (w0 + j), out);
                        }
                    }
                }
                tc::wait_st();
                tc::fence_before_sync();
                tc::arrive_warp(&s.k_full[st]);
            }
        });
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        const int r = 32 * quad + lane;
        uint4 c0, c1;
        uint32_t vs = 0, vz = 0;
        auto fetch = [&](size_t plane, int xt) {
            const int t = xt * kTile + r;
            if (xt < a.nt_packed && t < a.n_packed) {
                const uint4 *src = reinterpret_cast<const uint4 *>(a.v_codes + (plane * a.cap + t) * 8);
                c0 = __ldg(src);
                c1 = __ldg(src + 1);
                vs = __ldg(a.v_scale + plane * a.cap + t);
                vz = __ldg(a.v_zero + plane * a.cap + t);
            }
        };
        segments([&](const Seg &sg) { fetch(sg.kvh, sg.x0); }, [&](const Seg &sg) {
            // ---------------- V: token 32 quad + lane of the tile
            const size_t plane = (size_t)sg.kvh;
            const Offset off(lane & 1);
            for (int i = 0; i < sg.n; ++i) {
                const int k = it + i, st = k & 1, xt = sg.x0 + i;
                const bool packed = xt < a.nt_packed;
                const int t = (packed ? xt : xt - a.nt_packed) * kTile + r;
                uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                const bool live = t < (packed ? a.n_packed : a.n_res);
                // a token that is not there is zero everywhere: P = 0 must not meet garbage
                const uint32_t s2 = vs * 0x00010001u;
                const float zs = live && packed ? fmaf(lane & 1 ? 2.f : 1.f, h2f((uint16_t)vs), h2f((uint16_t)vz)) : 0.f;
                const uint16_t zh = f2h(zs), zl = f2h(zs - h2f(zh));
                fetch(plane, xt + 1);
                if (k >= 2 && !wait_warp(s, &s.o_done[st], ph_prev(k))) break;
                reinterpret_cast<uint16_t *>(s.vz[st][0])[r] = zh;
                reinterpret_cast<uint16_t *>(s.vz[st][1])[r] = zl;
                unsigned char *row = reinterpret_cast<unsigned char *>(s.v[st][0]) + r * 128;
                auto put = [&](int wi, const uint32_t *out) {   // the row's 16-byte chunks 2 wi, 2 wi + 1
                    unsigned char *dst = row + (wi >> 2) * (kTile * 128);
                    const int ch = (2 * (wi & 3)) ^ (r & 7);
                    *reinterpret_cast<uint4 *>(dst + (ch << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
                    *reinterpret_cast<uint4 *>(dst + ((ch ^ 1) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
                };
                if (packed && live) {   // (one answer a warp: the packed tokens are a multiple of 32)
#pragma unroll 1
                    for (int wi = 0; wi < 8; wi += 2) {
                        uint32_t out[16];
                        dequant_word(w[0], off, [&](int) { return s2; }, out);
                        dequant_word(w[1], off, [&](int) { return s2; }, out + 8);
                        put(wi, out);
                        put(wi + 1, out + 8);
#pragma unroll
                        for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
                    }
                } else if (packed) {
                    const uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
                    for (int wi = 0; wi < 8; ++wi) put(wi, out);
                } else {
                    int slot = a.res_start + t;
                    if (slot >= a.ring) slot -= a.ring;
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.v_res + (plane * a.ring + (live ? slot : 0)) * kD);
#pragma unroll 1
                    for (int w0 = 0; w0 < 8; w0 += 2) {
                        uint4 x[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = __ldg(src + 2 * w0 + j);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t out[8];
                            pair_order(x[2 * j], x[2 * j + 1], out);
#pragma unroll
                            for (int e = 0; e < 8; ++e) out[e] = live ? hmul2(out[e], kHalf2) : 0u;
                            put(w0 + j, out);
                        }
                    }
                }
                tc::fence_proxy_async_smem();
                tc::arrive_warp(&s.v_full[st]);
            }
        });
    } else if (warp < 28) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        segments([&](const Seg &sg) { load_rows<N, 512>(s, a, sg, tid - 384); }, [&](const Seg &sg) {
            if (warp >= 12 + 4 * kP) return;
            // ---------------- softmax: token lane r, rows n0 .. n0 + C - 1
            const int half = (warp - 12) >> 2, n0 = half * C, r = 32 * quad + lane, bar = 1 + half;
            const float sc = 2.f * a.scale_log2;
            float *bias = s.bias[warp - 12];
            bool ok = true;
            for (int i = 0; i < sg.n; ++i) {
                const int k = it + i, st = k & 1, xt = sg.x0 + i;
                const bool live = xt < a.nt_packed ? xt * kTile + r < a.n_packed
                                                   : (xt - a.nt_packed) * kTile + r < a.n_res;
                // S and T of the tile; P, alpha and the flag of two tiles ago have been read
                ok = ok && wait_warp(s, &s.s_full[st], ph(k));
                tc::fence_after_sync();
                const uint32_t ts = tmem + lanes + kColS + st * N + n0;
                const unsigned long long sc2 = f2pack(sc, sc);
                // the tile's log2 scores relative to the references; a second time if these move
                float x[C];
                bool moved = false, aborted = false;
                for (;;) {
                    tc::tmem_ld<C>(ts, *reinterpret_cast<uint32_t(*)[C]>(&x[0]));
                    for (int j = lane; j < C; j += 32) bias[j] = s.tz[k & 3][quad][n0 + j] - s.m[n0 + j];
                    __syncwarp();
                    float mx0 = -INFINITY, mx1 = -INFINITY;
                    tc::wait_ld();
#pragma unroll
                    for (int j = 0; j < C; j += 4) {
                        const float4 b4 = *reinterpret_cast<const float4 *>(&bias[j]);
                        f2unpack(ffma2(f2pack(x[j], x[j + 1]), sc2, f2pack(b4.x, b4.y)), x[j], x[j + 1]);
                        f2unpack(ffma2(f2pack(x[j + 2], x[j + 3]), sc2, f2pack(b4.z, b4.w)), x[j + 2], x[j + 3]);
                        mx0 = max3(mx0, x[j], x[j + 1]);
                        mx1 = max3(mx1, x[j + 2], x[j + 3]);
                    }
                    // does a score pass its row's reference by kLazy?  (a failed wait joins the vote: the
                    // warps of a half leave the loop together, at this barrier)
                    if (moved || (i > 0 && !or_over(bar, !ok || (live && fmaxf(mx0, mx1) > kLazy)))) break;
                    moved = true;
                    if (or_over(bar, !ok)) {
                        ok = false;
                        aborted = true;
                        break;
                    }
                    // column maxima of the tile -> new references; the sums and O'^T follow
                    if (!live)
#pragma unroll
                        for (int j = 0; j < C; ++j) x[j] = -INFINITY;
                    col_max<C, 16>(x, lane);
                    s.wmax[quad][n0 + lane / (32 / C)] = x[0];
                    sync_half(bar);
                    if (r < C) {
                        const int n = n0 + r;
                        const float top = fmaxf(fmaxf(s.wmax[0][n], s.wmax[1][n]), fmaxf(s.wmax[2][n], s.wmax[3][n]));
                        // how far the reference moves; the first tile's maximum sets it
                        const float up = i > 0 ? fmaxf(top, 0.f) : top == -INFINITY ? 0.f : top;
                        s.m[n] += up;
                        s.alpha[st][n] = i > 0 ? ex2(-up) : 1.f;
                    }
                    sync_half(bar);
                    if (i > 0) {
                        ok = wait_warp(s, &s.o_done[(k - 1) & 1], ph(k - 1));
                        tc::fence_after_sync();
                        const uint32_t to = tmem + lanes + kColO + n0;
#pragma unroll 1
                        for (int j = 0; ok && j < C; j += 8) {
                            uint32_t o[8];
                            tc::tmem_ld<8>(to + j, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * s.alpha[st][n0 + j + e]);
                            tc::tmem_st<8>(to + j, o);
                        }
                        tc::wait_st();
                    }
                }
                if (!ok) {
                    if (aborted) break;
                    continue;   // to the next tile's vote, or the epilogue
                }
                if (r == 0) s.resc[st][half] = moved;
                const uint32_t live2 = live ? 0xffffffffu : 0u;
                unsigned char *row = reinterpret_cast<unsigned char *>(s.p[st][n0 >> 6]) + r * 128;
#pragma unroll
                for (int j = 0; j < C; j += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = pack_half2(ex2(x[j + 2 * e]), ex2(x[j + 2 * e + 1])) & live2;
                    *reinterpret_cast<uint4 *>(row + (((((n0 + j) & 63) >> 3) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                tc::fence_proxy_async_smem();
                tc::fence_before_sync();
                tc::arrive_warp(&s.p_full[st]);
            }
            // ---------------- epilogue: the segment's state to slot c + u
            const int last = it + sg.n - 1;
            if (ok) ok = wait_warp(s, &s.o_done[last & 1], ph(last));
            asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(5 + half), "n"(160) : "memory");   // the sums are in s.l, s.pz
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
                        if (j + e < rows)
                            base[(size_t)(n0 + j + e) * kPreStride + ch] = fmaf(2.f, __uint_as_float(o[e]), s.pz[n0 + j + e]);
                }
                if (r < rows) {
                    const int n = n0 + r;
                    base[(size_t)n * kPreStride + 128] = s.m[n];
                    base[(size_t)n * kPreStride + 129] = s.l[n];
                }
            }
            tc::fence_before_sync();
        });
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
        segments([](const Seg &) {}, [&](const Seg &sg) {
            // ---------------- sums over P: [1; hi; lo] P, rows g_ = 0, 1, 2 of the product, for rows n0 .. n0 + 8 NT - 1
            constexpr int NT = N / 8 / kSW;   // 8-row tiles of a warp
            constexpr int KB = NT < 2 ? 8 : 16 / NT;   // 16-token steps whose loads go out together
            if (quad < kSW) {
                const int n0 = quad * NT * 8, half = quad;
                float total[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j) total[j][0] = total[j][1] = 0.f;
                // ldmatrix rows: token (lane & 15) of a 16-token step; columns: an 8-row chunk of P (lanes
                // 16-31 the next one; with one chunk in all the same one again)
                const int trow = lane & 15, ch0 = ((n0 & 63) >> 3) + (NT > 1 ? lane >> 4 : 0);
                for (int i = 0; i < sg.n; ++i) {
                    const int k = it + i, st = k & 1;
                    if (!wait_warp(s, &s.v_full[st], ph(k)) || !wait_warp(s, &s.p_full[st], ph(k))) break;
                    if (s.resc[st][half]) {
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const float2 al = *reinterpret_cast<const float2 *>(&s.alpha[st][n0 + 8 * j + 2 * t_]);
                            total[j][0] *= al.x;
                            total[j][1] *= al.y;
                        }
                    }
                    float d[NT][4];   // this tile's sums (a long sum stays in fp32 additions)
#pragma unroll
                    for (int j = 0; j < NT; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
                    const uint32_t *zrow = s.vz[st][g_ == 2] + t_;
                    const uint32_t one = g_ == 0 ? 0x3C003C00u : 0u, zmask = g_ == 1 || g_ == 2 ? 0xffffffffu : 0u;
                    const uint32_t prow = smem_addr(s.p[st][n0 >> 6]) + trow * 128;
#pragma unroll 1
                    for (int k0 = 0; k0 < 8; k0 += KB) {
                        uint32_t af[KB][2], b[KB][(NT + 1) / 2][4];
#pragma unroll
                        for (int e = 0; e < KB; ++e) {
                            af[e][0] = (zrow[8 * (k0 + e)] & zmask) | one;
                            af[e][1] = (zrow[8 * (k0 + e) + 4] & zmask) | one;
#pragma unroll
                            for (int j = 0; j < NT; j += 2)
                                ldmatrix_x4_t(b[e][j / 2], prow + (k0 + e) * 2048 + (((ch0 + j) ^ (trow & 7)) << 4));
                        }
#pragma unroll
                        for (int e = 0; e < KB; ++e) {
                            const uint32_t a4[4] = {af[e][0], 0u, af[e][1], 0u};
#pragma unroll
                            for (int j = 0; j < NT; j += 2) {
                                mma16816(d[j], a4, b[e][j / 2][0], b[e][j / 2][1]);
                                if (NT > 1) mma16816(d[j + (NT > 1)], a4, b[e][j / 2][2], b[e][j / 2][3]);
                            }
                        }
                    }
                    tc::arrive_warp(&s.o_done[st]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        total[j][0] += d[j][0];
                        total[j][1] += d[j][1];
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float lo_part = __shfl_down_sync(0xffffffffu, total[j][e], 4);   // row g_ + 1
                        const int n = n0 + 8 * j + 2 * t_ + e;
                        if (g_ == 0) s.l[n] = total[j][e];
                        if (g_ == 1) s.pz[n] = total[j][e] + lo_part;
                    }
                }
                __syncwarp();
                asm volatile("barrier.cta.arrive %0, %1;\n" ::"r"(5 + half), "n"(160) : "memory");   // to the half's epilogue
            }
        });
    }
    if (warp == 1 || warp == 3) {   // every MMA issued has finished (after an expired wait, too)
        if (tc::elect_one()) tc::commit(&s.drain[warp >> 1]);
        __syncwarp();
        mbar_wait(&s.drain[warp >> 1], 0);
    }
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, kCols);
    // (words of CTAs that this call does not have: zero)
    if (tid < kMaxCtas && tid % a.tab.P == c) a.status[tid] = tid == c && s.abort ? 1u : 0u;
}

std::mutex g_mu;
bool g_attr[kMaxDevices] = {};
int g_sms[kMaxDevices] = {};

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

int prefix_launch(const PrefixCall &call, int B, const uint16_t *q, int Hq, float sm_scale, cudaStream_t stream,
                  PreTab *tab) {
    const minikv_cache *p = call.prefix;
    const int *shared = call.shared;
    void *ws = call.ws;
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
