// gdn_chunk.cu -- the gated delta rule over packed chunks of new tokens, from
// the states of a pool and back into it.
//
// Per value head (key head h / (Hv/Hk)) the state S is dv x dk, and a token makes
// S <- a S + u k^T, u = b (v - a S k), a = exp(g), and reads o = S q.  Over a block
// of C = 64 tokens behind S_0, with G the running sum of g in the block:
//   (I + A) U = diag(b) (V - diag(e^G) K S_0^T),  A_ij = b_i e^(G_i - G_j) k_i.k_j  (j < i)
//   O   = diag(e^G) Q S_0^T + P U,                P_ij = e^(G_i - G_j) q_i.k_j      (j <= i)
//   S_C = e^(G_C) S_0 + (diag(e^(G_C - G)) U)^T K
// With T = (I + A)^-1 these are products, all of them on the tensor cores.
//
// What bounds it: blocks of one sequence follow one another, and in each a chain
// of three products and the register work between them; sequences, heads and 128
// rows of a state each have a CTA.
//  * Everything is held transposed, a row of the state (and of U, O) per lane of
//    tensor memory: X = S K^T, then R = b (v - e^G X) becomes U = R T^T, U becomes
//    S' = U~ K, and each result is read by the threads that hold its rows and written
//    back as the next product's first operand, in tensor memory.  Two threads share
//    a row; S itself stays in their registers, in fp32.
//  * Eight warps run that chain; four prepare the next block meanwhile: keys and
//    queries to fp16, K K^T and Q K^T on the tensor cores, decays, the inverse T.
//  * Products take fp16 operands and fp32 sums.  S, R, U and T are fp32 values held
//    as two fp16 parts (x = hi + lo, 2^-22 of x), so that a state stays an fp32 one; what only an
//    output sees (S and U there, P and the decayed queries) is one part, 2^-11 beside
//    the output's own 2^-8.  (bf16 parts would need three for that, half as many
//    products again.)
//  * fp16 reaches from 2^-24 to 2^16, so everything is scaled by powers of two, exactly:
//    a key to a largest element in [2^-4, 2^-3) (k = 2^e k': b' = 4^e b, v' = 2^-e v,
//    u' = 2^e u is the same rule), a query likewise, and a row of S, R and U by one
//    factor a block, from bounds of what it can reach: with b |k|^2 <= 2 a token adds
//    at most |b' v'| |k'| to a row's norm, and |k'| is from 2^-4 to sqrt(2), so that u' <=
//    32 |S| + |b' v'|: |S| <= 2^6 and |b' v'| <= 2^3 at a block's start keep all of it
//    below 2^16, and the parts are off by 2^-27 of the larger of the two at most.
//  * The inverse: four 16 x 16 blocks by forward substitution, then joined twice by
//    -T22 (A21 T11), in fp32 on the CUDA cores, which is as stable as the substitution.
//  * G is summed in 64 bits and its differences are taken of two fp32 parts: a gate that
//    closes (g = -1000) leaves the decays behind it exact.
#include "gdn_pool.cuh"
#include "tcgen05.cuh"

namespace sv {
namespace gdn {
namespace {

constexpr int C = 64;        // tokens of a block
constexpr int ROWS = 128;    // rows of the state a CTA holds (TMEM lanes)
constexpr int CHAIN = 256, PREP = 128, THREADS = CHAIN + PREP;
constexpr int AS = 68;       // row stride of the inverse's fp32 matrices
constexpr int MAX_SORTED = 128;
constexpr float G_LEAST = -10000.f;  // e^g is 0 long before
constexpr float Q_GAIN = 1024.f;     // queries and P are taken so much larger: e^G down to 2^-24 keeps its bits

// One block's scalars.
struct Scalars {
  float bv[C], bx[C], en[C], os[C];  // of v in R, of X in R, of U in U~, of the output
  float gc;                          // decay over the block
  float pad[3];
};

template <int DK>
struct L {
  static constexpr int G = DK / 64;                  // 64-column groups
  static constexpr int KQ_BYTES = G * 128 * 128;     // K' in rows 0..63, Q' in 64..127
  static constexpr int RAW_BYTES = 128 * DK * 2;
  static constexpr int V_BYTES = C * ROWS * 2;
  static constexpr int T_BYTES = C * 128;            // one part; P too
  static constexpr int KQ = 1024;                    // [2]
  static constexpr int T = KQ + 2 * KQ_BYTES;        // [2][hi, lo]
  static constexpr int P = T + 4 * T_BYTES;          // [2]
  static constexpr int V = P + 2 * T_BYTES;          // [3]
  static constexpr int RAW = V + 3 * V_BYTES;
  static constexpr int A = RAW + RAW_BYTES;          // fp32 [64][AS], inverted in place
  static constexpr int SC = A + C * AS * 4;          // Scalars[2]
  static constexpr int GH = SC + 2 * (int)sizeof(Scalars);  // G in units of log 2, two parts [2][64]
  static constexpr int EXP = GH + 2 * C * 4;         // exponent of a key's or query's scale [128]
  static constexpr int XCHG = EXP + 128 * 4;         // [2][2][ROWS]
  static constexpr int BYTES = XCHG + 4 * ROWS * 4;
  static_assert(BYTES <= 227 * 1024, "shared memory");
  // tensor memory: S in two parts; X, then U beside it, then S' over both; R in two
  // parts, then U~ in two and U in one; O; K K^T over Q K^T
  static constexpr uint32_t SH = 0, SL = DK / 2, X = 128, U = 192, D = 128, R = 256, O = 352, KK = 416;
};

struct ChunkParams {
  PoolParams p;
  int blocks;  // of ROWS rows a head
  int stall;   // test aid: the first block's keys never arrive
};

__device__ __forceinline__ uint32_t swz(int row, int c16) {  // 16-byte piece c16 of a 128-byte row
  return (uint32_t)(row * 128 + ((c16 ^ (row & 7)) << 4));
}

// Two fp32 values as fp16 parts.
__device__ __forceinline__ void split2(f2 x, uint32_t &hi, uint32_t &lo) {
  const float2 v = unpack2(x);
  hi = pack_f16x2(v.x, v.y);
  const float2 r = unpack2(fma2(pack2(f16lo(hi), f16hi(hi)), pack2(-1.f, -1.f), x));
  lo = pack_f16x2(r.x, r.y);
}

__device__ __forceinline__ float pow2_field(int e) { return __int_as_float(e << 23); }  // 2^(e - 127)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

template <int DK>
__global__ void __launch_bounds__(THREADS, 1) chunk_kernel(const ChunkParams CP) {
  using Y = L<DK>;
  const PoolParams &P = CP.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // swizzled tiles need it; so it is in a kernel without static shared memory
    if (threadIdx.x == 0) atomicOr(P.err, ERR_TIMEOUT);
    return;
  }
  uint64_t *kq_full = reinterpret_cast<uint64_t *>(smem);  // [2] keys, queries and values of a block
  uint64_t *tp_full = kq_full + 2;                         // [2] T, P, decayed queries, scalars
  uint64_t *free_ = tp_full + 2;                           // [2] all of a block's read
  uint64_t *x_done = free_ + 2, *u_done = x_done + 1, *d_done = u_done + 1, *o_done = d_done + 1;
  uint64_t *k_done = o_done + 1, *idle = k_done + 1;       // idle [2]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(idle + 2);
  int *pick = reinterpret_cast<int *>(tmem_slot + 1);
  Scalars *sc_all = reinterpret_cast<Scalars *>(smem + Y::SC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kq_full[i], 4 + (i == 0 ? CP.stall : 0));
      mbar_init(&tp_full[i], 4);
      mbar_init(&free_[i], 9);
      mbar_init(&idle[i], 1);
    }
    for (uint64_t *b : {x_done, u_done, d_done, o_done, k_done}) mbar_init(b, 1);
    fence_barrier_init();
    *pick = 0;
  }
  if (warp == 8) {
    tc::tmem_alloc(tmem_slot, 512u);
    tc::tmem_relinquish();
  }
  pdl_wait();
  // ---- the item: longest sequences first ----
  const int per = P.Hv * CP.blocks;
  int b = blockIdx.x / per;
  const int rest = blockIdx.x - b * per, h = rest / CP.blocks, i0 = (rest - h * CP.blocks) * ROWS;
  __syncthreads();
  if (P.B > 1 && P.B <= MAX_SORTED) {
    int *len = reinterpret_cast<int *>(smem + Y::GH);  // (GH and EXP are 256 ints)
    if (tid < P.B) len[tid] = rows_of(P, tid, false).y;
    __syncthreads();
    if (tid < P.B) {
      int rank = 0;
      const int mine = len[tid];
      for (int i = 0; i < P.B; ++i) rank += len[i] > mine || (len[i] == mine && i < tid) ? 1 : 0;
      if (rank == b) *pick = tid;
    }
    __syncthreads();
    b = *pick;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const bool report = rest == 0 && tid == 0;
  const int2 own = rows_of(P, b, report);
  const int slot = slot_of(P, b, report);
  const int n = (own.y + C - 1) / C;  // blocks
  const int hk = h / (P.Hv / P.Hk);

  if (warp >= 8) {
    // ------------------------------------------------ the next block --
    // 384 threads start with 168 registers each: 256 * 184 + 128 * 136 is the same total
    setmaxnreg_dec<136>();
    const int pt = tid - CHAIN, pw = warp - 8;
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(P.k.ptr) + (long long)hk * P.k.head_stride;
    const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(P.q.ptr) + (long long)hk * P.q.head_stride;
    const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(P.v.ptr) + (long long)h * P.v.head_stride + i0;
    const int live = imin(ROWS, P.dv - i0);  // rows of the state that exist
    float *A = reinterpret_cast<float *>(smem + Y::A);
    float *gh = reinterpret_cast<float *>(smem + Y::GH), *gl = gh + C;
    int *ex = reinterpret_cast<int *>(smem + Y::EXP);
    const bool issuer = pw == 0 && tc::elect_one();
    const uint32_t lane_off = (uint32_t)(pw * 32) << 16;
    auto bar = [&]() { named_barrier(1, PREP); };
    // Copies of block c: keys and queries as they are, values to their place.
    auto fetch = [&](int c) {
      const int m = imin(C, own.y - c * C);
      const long long r0 = own.x + (long long)c * C;
      const uint32_t raw = smem_u32(smem + Y::RAW), vs = smem_u32(smem + Y::V + (c % 3) * Y::V_BYTES);
      constexpr int PC = DK / 8;
#pragma unroll 4
      for (int e = pt; e < 128 * PC; e += PREP) {
        const int r = e / PC, x = e % PC, t = r & 63;
        const bool in = t < m;
        const __nv_bfloat16 *src = r < C ? kp + (r0 + (in ? t : 0)) * P.k.token_stride : qp + (r0 + (in ? t : 0)) * P.q.token_stride;
        cp_async16(raw + r * DK * 2 + ((x ^ (r & 7)) << 4), src + x * 8, in);
      }
#pragma unroll 4
      for (int e = pt; e < C * (ROWS / 8); e += PREP) {
        const int t = e / (ROWS / 8), x = e % (ROWS / 8);
        const __nv_bfloat16 *src = vp + (r0 + (t < m ? t : 0)) * P.v.token_stride;
        const uint32_t at = vs + t * ROWS * 2 + x * 16;
        if (x * 8 + 8 <= live || x * 8 >= live || t >= m) {
          const bool in = t < m && x * 8 < live;
          cp_async16(at, in ? src + x * 8 : src, in);
        } else {  // the last columns, fewer than eight: nothing behind them is read
          __nv_bfloat16 *d = reinterpret_cast<__nv_bfloat16 *>(smem + Y::V + (c % 3) * Y::V_BYTES) + t * ROWS + x * 8;
          for (int y = 0; y < 8; ++y) d[y] = x * 8 + y < live ? src[x * 8 + y] : __float2bfloat16_rn(0.f);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    bool ok = true;
    if (n > 0) fetch(0);
    for (int c = 0; c < n; ++c) {
      const int st = c & 1, m = imin(C, own.y - c * C);
      Scalars &S = sc_all[st];
      // gates of two tokens a lane (first warp)
      float g0 = 0.f, g1 = 0.f, be = 0.f;
      const long long r0 = own.x + (long long)c * C;
      if (pw == 0) {
        if (2 * lane < m) g0 = P.g[(r0 + 2 * lane) * P.Hv + h];
        if (2 * lane + 1 < m) g1 = P.g[(r0 + 2 * lane + 1) * P.Hv + h];
      }
      if (pt < m && pt < C) be = P.b[(r0 + pt) * P.Hv + h];
      if (c >= 2 && ok) ok = mbar_wait(&free_[st], ((c >> 1) - 1) & 1, P.err);
      cp_async_wait_all();
      fence_proxy_async();
      bar();
      uint8_t *kq = smem + Y::KQ + st * Y::KQ_BYTES;
      // keys and queries to fp16: eight threads a row, DK/8 elements each
      constexpr int PR = DK / 64;  // 16-byte pieces a thread
#pragma unroll 2
      for (int r = pt >> 3; r < 128; r += PREP / 8) {
        const int s8 = pt & 7;
        uint4 w[PR];
        uint32_t mx = 0;
#pragma unroll
        for (int y = 0; y < PR; ++y) {
          const int x = s8 + 8 * y;
          w[y] = *reinterpret_cast<const uint4 *>(smem + Y::RAW + r * DK * 2 + ((x ^ (r & 7)) << 4));
#pragma unroll
          for (int z = 0; z < 4; ++z) {  // (of finite values the larger has the larger bits)
            const uint32_t v = (&w[y].x)[z];
            mx = max(mx, max(v & 0x7fffu, (v >> 16) & 0x7fffu));
          }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int E = (int)(mx >> 7);
        const float f = pow2_field(imax(250 - E, 1));
        const f2 f2x = pack2(f, f);
#pragma unroll
        for (int y = 0; y < PR; ++y) {
          const int x = s8 + 8 * y;
          uint4 d;
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint32_t v = (&w[y].x)[z];
            const float2 p = unpack2(mul2(pack2(bf16lo(v), bf16hi(v)), f2x));
            (&d.x)[z] = pack_f16x2(p.x, p.y);
          }
          *reinterpret_cast<uint4 *>(kq + (x >> 3) * 128 * 128 + swz(r, x & 7)) = d;
        }
        if (s8 == 0) ex[r] = E;
      }
      if (pw == 0) {  // running sums of the gates, in units of log 2
        double a0 = (double)(g0 < G_LEAST ? G_LEAST : g0), a1 = a0 + (double)(g1 < G_LEAST ? G_LEAST : g1);
        double x = a1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const double k2 = 1.4426950408889634074;
        const double s1 = x * k2, s0 = (x - a1 + a0) * k2;
        gh[2 * lane] = (float)s0, gl[2 * lane] = (float)(s0 - (double)(float)s0);
        gh[2 * lane + 1] = (float)s1, gl[2 * lane + 1] = (float)(s1 - (double)(float)s1);
      }
      fence_proxy_async();
      bar();
      if (issuer && ok) {
        const uint64_t da = tc::smem_desc_sw128(smem_u32(kq), 16, 1024);
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const uint64_t d = da + ((ks >> 2) * 128 * 128 + (ks & 3) * 32) / 16;
          tc::mma_bf16(tb + Y::KK, d, d, tc::idesc_f16_f32(128, C, false), ks > 0);
        }
        tc::commit(k_done);
      }
      __syncwarp();
      if (pt < C) {
        const float gt = gh[pt] + gl[pt];
        const float e1 = pow2_field(imin(ex[pt] + 4, 254));  // 2^e
        const float ga = ex2_approx(gt), bs = be * e1;
        S.bv[pt] = bs;
        S.bx[pt] = bs * e1 * ga;
        S.en[pt] = ex2_approx((gh[C - 1] - gh[pt]) + (gl[C - 1] - gl[pt]));
        S.os[pt] = pow2_field(imin(ex[C + pt] + 4, 254)) * (1.f / Q_GAIN);
        if (pt == C - 1) S.gc = ga;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&kq_full[st]);
      if (c + 1 < n) fetch(c + 1);
      if (ok) ok = mbar_wait(k_done, c & 1, P.err);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      // ---- A (rows 0..63) and P (64..127) ----
      {
        const int i = (pw & 1) * 32 + lane;
        const bool isP = pw >= 2;
        const float hi_i = gh[i], lo_i = gl[i];
        const float f = isP ? Q_GAIN : pow2_field(imin(ex[i] + 4, 254));
        // b' of this row (b is with the thread of the token)
        float bi = 1.f;
        if (!isP) bi = be * f * f;  // pt == i here
        const f2 rowf = pack2(isP ? Q_GAIN : bi, isP ? Q_GAIN : bi), hi2 = pack2(hi_i, hi_i), lo2 = pack2(lo_i, lo_i);
        const f2 neg = pack2(-1.f, -1.f);
        uint8_t *pp = smem + Y::P + st * Y::T_BYTES;
#pragma unroll
        for (int c0 = 0; c0 < 2; ++c0) {
          uint32_t raw[32];
          const bool any = c0 == 0 || (pw & 1);  // columns 32.. of rows 0..31 are zero
          if (any && ok) {
            tc::ld32(tb + Y::KK + c0 * 32 + lane_off, raw);
            tc::wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float y[8];
#pragma unroll
            for (int z = 0; z < 8; z += 4) {
              const int j = c0 * 32 + e + z;
              const ulonglong2 hj = *reinterpret_cast<const ulonglong2 *>(gh + j), lj = *reinterpret_cast<const ulonglong2 *>(gl + j);
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const f2 dh = fma2(w ? hj.y : hj.x, neg, hi2), dl = fma2(w ? lj.y : lj.x, neg, lo2);
                const float2 d = unpack2(add2(dh, dl));
                const f2 kk = pack2(__uint_as_float(raw[e + z + 2 * w]), __uint_as_float(raw[e + z + 2 * w + 1]));
                const float2 t = unpack2(mul2(mul2(kk, rowf), pack2(ex2_approx(d.x), ex2_approx(d.y))));
                const int jj = j + 2 * w;
                y[z + 2 * w] = any && (isP ? jj <= i : jj < i) ? t.x : 0.f;
                y[z + 2 * w + 1] = any && (isP ? jj + 1 <= i : jj + 1 < i) ? t.y : 0.f;
              }
            }
            const int j = c0 * 32 + e;
            if (isP) {
              *reinterpret_cast<uint4 *>(pp + swz(i, j >> 3)) = make_uint4(pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3]),
                                                                          pack_f16x2(y[4], y[5]), pack_f16x2(y[6], y[7]));
            } else {
              *reinterpret_cast<float4 *>(A + i * AS + j) = make_float4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<float4 *>(A + i * AS + j + 4) = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
        }
      }
      tc::fence_before_sync();
      bar();
      // ---- decayed queries (their product with the keys is done) ----
#pragma unroll 2
      for (int r = C + (pt >> 3); r < 128; r += PREP / 8) {
        const __half2 ga = __float2half2_rn(ex2_approx(gh[r - C] + gl[r - C]) * Q_GAIN);
#pragma unroll
        for (int y = 0; y < PR; ++y) {
          uint4 *p = reinterpret_cast<uint4 *>(kq + y * 128 * 128 + swz(r, pt & 7));
          uint4 d = *p;
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            __half2 v = *reinterpret_cast<__half2 *>(&(&d.x)[z]);
            v = __hmul2(v, ga);
            (&d.x)[z] = *reinterpret_cast<uint32_t *>(&v);
          }
          *p = d;
        }
      }
      // ---- T = (I + A)^-1 in place: a 16 x 16 block a warp, a column a lane ----
      {
        const int o = pw * 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
          for (int j = 0; j < i; ++j) {
            const float a = A[(o + i) * AS + o + j];
            if (j & 1) s1 = fmaf(-a, x[j], s1); else s0 = fmaf(-a, x[j], s0);
          }
          x[i] = s0 + s1;
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) A[(o + i) * AS + o + lane] = x[i];
        }
      }
      bar();
      // joined: T21 = -T22 (A21 T11), 16 rows and columns of two pairs, then 32 of one
      {
        // one row, four columns a thread: pair pt / 64
        const int o = (pt >> 6) * 32, i = o + 16 + ((pt & 63) >> 2), j = o + (pt & 3) * 4;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
          f2 w0 = 0, w1 = 0;
          const int k0 = o + 16 * pass;
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(A + i * AS + k0 + k);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const ulonglong2 t = *reinterpret_cast<const ulonglong2 *>(A + (k0 + k + z) * AS + j);
              const float av = pass ? -(&a.x)[z] : (&a.x)[z];
              w0 = fma2(pack2(av, av), t.x, w0), w1 = fma2(pack2(av, av), t.y, w1);
            }
          }
          bar();
          *reinterpret_cast<ulonglong2 *>(A + i * AS + j) = make_ulonglong2(w0, w1);
          bar();
        }
      }
      {
        const int i = 32 + (pt >> 3) * 2, j = (pt & 7) * 4;  // two rows, four columns
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
          f2 w[2][2] = {{0, 0}, {0, 0}};
          const int k0 = 32 * pass;
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(A + i * AS + k0 + k);
            const float4 a1 = *reinterpret_cast<const float4 *>(A + (i + 1) * AS + k0 + k);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const ulonglong2 t = *reinterpret_cast<const ulonglong2 *>(A + (k0 + k + z) * AS + j);
              const float p = pass ? -(&a.x)[z] : (&a.x)[z], q = pass ? -(&a1.x)[z] : (&a1.x)[z];
              w[0][0] = fma2(pack2(p, p), t.x, w[0][0]), w[0][1] = fma2(pack2(p, p), t.y, w[0][1]);
              w[1][0] = fma2(pack2(q, q), t.x, w[1][0]), w[1][1] = fma2(pack2(q, q), t.y, w[1][1]);
            }
          }
          bar();
          *reinterpret_cast<ulonglong2 *>(A + i * AS + j) = make_ulonglong2(w[0][0], w[0][1]);
          *reinterpret_cast<ulonglong2 *>(A + (i + 1) * AS + j) = make_ulonglong2(w[1][0], w[1][1]);
          bar();
        }
      }
      // ---- T in two parts: half a row a thread ----
      {
        const int i = pt >> 1, j0 = (pt & 1) * 32;
        uint8_t *th = smem + Y::T + st * 2 * Y::T_BYTES, *tl = th + Y::T_BYTES;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint4 hi, lo;
          const int j = j0 + e;
          const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(A + i * AS + j), d = *reinterpret_cast<const ulonglong2 *>(A + i * AS + j + 4);
          split2(a.x, hi.x, lo.x);
          split2(a.y, hi.y, lo.y);
          split2(d.x, hi.z, lo.z);
          split2(d.y, hi.w, lo.w);
          *reinterpret_cast<uint4 *>(th + swz(i, j >> 3)) = hi;
          *reinterpret_cast<uint4 *>(tl + swz(i, j >> 3)) = lo;
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tp_full[st]);
    }
    cp_async_wait_all();
    if (issuer) {
      tc::commit(&idle[0]);
      spin_wait(&idle[0], 0, P.err);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------- the chain --
    setmaxnreg_inc<184>();
    constexpr int SC = DK / 2;  // columns of S that are this thread's
    const int hf = warp >> 2, r = (warp & 3) * 32 + lane, i = i0 + r;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const bool live = i < P.dv;
    const bool issuer = warp == 0 && tc::elect_one();
    auto bar = [&]() { named_barrier(2, CHAIN); };
    float *xchg = reinterpret_cast<float *>(smem + Y::XCHG);
    uint32_t trades = 0;
    // the larger of a value that both threads of a row have
    auto both = [&](float x) {
      float *at = xchg + (trades & 1) * 2 * ROWS;
      ++trades;
      at[hf * ROWS + r] = x;
      named_barrier(3 + (warp & 3), 64);
      return fmaxf(x, at[(hf ^ 1) * ROWS + r]);
    };
    float *srow = P.states.ptr + (slot >= 0 ? slot : 0) * P.states.slot_stride + ((long long)h * P.dv + (live ? i : 0)) * DK + hf * SC;
    const bool kept = slot >= 0 && live && n > 0;
    f2 S[SC / 2];
#pragma unroll
    for (int e = 0; e < SC / 2; e += 2) {
      ulonglong2 x = make_ulonglong2(0, 0);
      if (kept) x = *reinterpret_cast<const ulonglong2 *>(srow + 2 * e);
      S[e] = x.x, S[e + 1] = x.y;
    }
    auto row_max = [&]() {
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int e = 0; e < SC / 2; ++e) {
        const float2 x = unpack2(S[e]);
        m0 = fmaxf(m0, fabsf(x.x)), m1 = fmaxf(m1, fabsf(x.y));
      }
      return fmaxf(m0, m1);
    };
    // largest |b' v'| of this thread's half of block c
    auto v_max = [&](int c) {
      const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(smem + Y::V + (c % 3) * Y::V_BYTES) + hf * 32 * ROWS + r;
      const float *bv = &sc_all[c & 1].bv[hf * 32];
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int t = 0; t < 32; t += 4) {
        const float4 b4 = *reinterpret_cast<const float4 *>(bv + t);
        m0 = fmaxf(m0, fmaxf(fabsf(b4.x * __bfloat162float(v[t * ROWS])), fabsf(b4.y * __bfloat162float(v[(t + 1) * ROWS]))));
        m1 = fmaxf(m1, fmaxf(fabsf(b4.z * __bfloat162float(v[(t + 2) * ROWS])), fabsf(b4.w * __bfloat162float(v[(t + 3) * ROWS]))));
      }
      return fmaxf(m0, m1);
    };
    // scale of a row: 2^-k with at most 1 behind it
    auto scale_of = [&](float most) { return pow2_field(253 - imin(imax(__float_as_int(most) >> 23, 27), 226)); };
    auto put_state = [&](float sc) {
      const f2 sc2 = pack2(sc, sc);
#pragma unroll
      for (int g = 0; g < SC / 32; ++g) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) split2(mul2(S[16 * g + e], sc2), hi[e], lo[e]);
        tc::st16(tb + Y::SH + hf * (SC / 2) + 16 * g + lane_off, hi);
        tc::st16(tb + Y::SL + hf * (SC / 2) + 16 * g + lane_off, lo);
      }
      tc::wait_st();
      tc::fence_before_sync();
    };
    bool ok = true;
    auto wait = [&](uint64_t *bar_, uint32_t parity) {
      if (ok) ok = spin_wait(bar_, parity, P.err);
      ok = __all_sync(0xffffffffu, ok);
    };
    float m = row_max();
    float sc = 1.f, isc_before = 1.f;
    if (n > 0) {
      wait(&kq_full[0], 0);
      sc = scale_of(both(fmaxf(m * 0.015625f, 0.125f * v_max(0))));
      put_state(sc);
      bar();
    }
    // O of block c
    auto put_out = [&](int c, float isc) {
      wait(o_done, c & 1);
      tc::fence_after_sync();
      const Scalars &Z = sc_all[c & 1];
      uint32_t raw[32];
      if (ok) {
        tc::ld32(tb + Y::O + hf * 32 + lane_off, raw);
        tc::wait_ld();
      }
      const int t0 = c * C + hf * 32, mt = imin(32, own.y - t0);
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(P.o.ptr) + (own.x + (long long)t0) * P.o.token_stride + (long long)h * P.o.head_stride + i;
#pragma unroll
      for (int t = 0; t < 32; ++t) {
        const float x = __uint_as_float(raw[t]) * isc * Z.os[hf * 32 + t];
        if (live && ok && t < mt) out[(long long)t * P.o.token_stride] = __float2bfloat16_rn(x);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&free_[c & 1]);
    };
    constexpr uint32_t IDN = tc::idesc_f16_f32(128, C, false), IDD = tc::idesc_f16_f32(128, DK, true);
    for (int c = 0; c < n; ++c) {
      const int st = c & 1;
      const uint32_t par = c & 1;
      const Scalars &Z = sc_all[st];
      const uint64_t dk = tc::smem_desc_sw128(smem_u32(smem + Y::KQ + st * Y::KQ_BYTES), 16, 1024);
      const uint64_t dkt = tc::smem_desc_sw128(smem_u32(smem + Y::KQ + st * Y::KQ_BYTES), 128 * 128, 1024);
      const uint64_t dt = tc::smem_desc_sw128(smem_u32(smem + Y::T + st * 2 * Y::T_BYTES), 16, 1024);
      const uint64_t dp = tc::smem_desc_sw128(smem_u32(smem + Y::P + st * Y::T_BYTES), 16, 1024);
      auto k_step = [](int ks) { return (uint64_t)(((ks >> 2) * 128 * 128 + (ks & 3) * 32) / 16); };
      // X = S K^T
      if (issuer && ok) {
        tc::fence_after_sync();
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            tc::mma_bf16_ts(tb + Y::X, tb + (p ? Y::SL : Y::SH) + ks * 8, dk + k_step(ks), IDN, p > 0 || ks > 0);
        tc::commit(x_done);
      }
      __syncwarp();
      if (c > 0) put_out(c - 1, isc_before);
      wait(&tp_full[st], (c >> 1) & 1);
      // R = b (v - e^G X)
      {
        const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(smem + Y::V + (c % 3) * Y::V_BYTES) + hf * 32 * ROWS + r;
        f2 vv[16];
        const f2 sc2 = pack2(sc, sc);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const f2 bv = *reinterpret_cast<const f2 *>(&Z.bv[hf * 32 + 2 * t]);
          vv[t] = mul2(mul2(pack2(__bfloat162float(v[2 * t * ROWS]), __bfloat162float(v[(2 * t + 1) * ROWS])), sc2), bv);
        }
        wait(x_done, par);
        tc::fence_after_sync();
        uint32_t raw[32];
        if (ok) {
          tc::ld32(tb + Y::X + hf * 32 + lane_off, raw);
          tc::wait_ld();
        }
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const f2 bx = mul2(*reinterpret_cast<const f2 *>(&Z.bx[hf * 32 + 2 * t]), pack2(-1.f, -1.f));
          split2(fma2(bx, pack2(__uint_as_float(raw[2 * t]), __uint_as_float(raw[2 * t + 1])), vv[t]), hi[t], lo[t]);
        }
        tc::st16(tb + Y::R + hf * 16 + lane_off, hi);
        tc::st16(tb + Y::R + 32 + hf * 16 + lane_off, lo);
        tc::wait_st();
        tc::fence_before_sync();
        bar();
      }
      // U = R T^T, and O = S Q^T
      if (issuer && ok) {
        tc::fence_after_sync();
#pragma unroll
        for (int p = 0; p < 3; ++p)  // hi hi, lo hi, hi lo
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
            tc::mma_bf16_ts(tb + Y::U, tb + Y::R + (p == 1 ? 32 : 0) + ks * 8, dt + (uint64_t)(((p == 2 ? Y::T_BYTES : 0) + ks * 32) / 16),
                            IDN, p > 0 || ks > 0);
        tc::commit(u_done);
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks)
          tc::mma_bf16_ts(tb + Y::O, tb + Y::SH + ks * 8, dk + k_step(ks) + 64 * 128 / 16, IDN, ks > 0);
      }
      __syncwarp();
      float um = 0.f;
      {
        f2 en[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) en[t] = *reinterpret_cast<const f2 *>(&Z.en[hf * 32 + 2 * t]);
        wait(u_done, par);
        tc::fence_after_sync();
        uint32_t raw[32];
        if (ok) {
          tc::ld32(tb + Y::U + hf * 32 + lane_off, raw);
          tc::wait_ld();
        }
        uint32_t hi[16], lo[16], u[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const float a = __uint_as_float(raw[2 * t]), d = __uint_as_float(raw[2 * t + 1]);
          u[t] = pack_f16x2(a, d);
          const f2 x = mul2(pack2(a, d), en[t]);
          const float2 y = unpack2(x);
          um = fmaxf(um, fmaxf(fabsf(y.x), fabsf(y.y)));
          split2(x, hi[t], lo[t]);
        }
        tc::st16(tb + Y::R + hf * 16 + lane_off, hi);
        tc::st16(tb + Y::R + 32 + hf * 16 + lane_off, lo);
        tc::st16(tb + Y::R + 64 + hf * 16 + lane_off, u);
        tc::wait_st();
        tc::fence_before_sync();
        bar();
      }
      // S' = U~ K, then O += P U
      if (issuer && ok) {
        tc::fence_after_sync();
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
            tc::mma_bf16_ts(tb + Y::D, tb + Y::R + p * 32 + ks * 8, dkt + (uint64_t)(ks * 2048 / 16), IDD, p > 0 || ks > 0);
        tc::commit(d_done);
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks)
          tc::mma_bf16_ts(tb + Y::O, tb + Y::R + 64 + ks * 8, dp + (uint64_t)(ks * 32 / 16), IDN, true);
        tc::commit(o_done);
        tc::commit(&free_[st]);
      }
      __syncwarp();
      const float gc = Z.gc, isc = 1.f / sc;  // (exact)
      float sc_next = sc;
      if (c + 1 < n) {
        wait(&kq_full[st ^ 1], ((c + 1) >> 1) & 1);
        // elements of k' are below 2^-3, 64 tokens: |S'| <= 8 |U~|; twice for the other half's
        sc_next = scale_of(both(fmaxf((gc * m + 8.f * um * isc) * 0.03125f, 0.125f * v_max(c + 1))));
      }
      {
        const f2 gc2 = pack2(gc, gc), isc2 = pack2(isc, isc);
#pragma unroll
        for (int e = 0; e < SC / 2; ++e) S[e] = mul2(S[e], gc2);
        wait(d_done, par);
        tc::fence_after_sync();
#pragma unroll
        for (int g = 0; g < SC / 32; ++g) {
          uint32_t raw[32];
          if (ok) {
            tc::ld32(tb + Y::D + hf * SC + 32 * g + lane_off, raw);
            tc::wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            S[16 * g + e] = fma2(pack2(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1])), isc2, S[16 * g + e]);
        }
      }
      put_state(sc_next);
      bar();
      m = row_max();
      isc_before = isc;
      sc = sc_next;
    }
    if (n > 0) put_out(n - 1, isc_before);
    if (kept && ok) {
#pragma unroll
      for (int e = 0; e < SC / 2; e += 2) *reinterpret_cast<ulonglong2 *>(srow + 2 * e) = make_ulonglong2(S[e], S[e + 1]);
    }
    if (issuer) {
      tc::commit(&idle[1]);
      spin_wait(&idle[1], 0, P.err);
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, 512u);
  }
}

template <int DK>
sv_status run_chunks(ChunkParams &CP, cudaStream_t s) {
  const long long items = (long long)CP.p.B * CP.p.Hv * CP.blocks;
  if (items > 0x7fffffffLL) return SV_ERR_UNSUPPORTED;
  return from_cuda(launch_early(chunk_kernel<DK>, dim3((unsigned)items), dim3(THREADS), (size_t)L<DK>::BYTES, s, CP));
}

}  // namespace
}  // namespace gdn
}  // namespace sv

using namespace sv;

extern "C" {

size_t gdn_chunk_workspace_bytes(int B, int T, int Hk, int Hv, int dk, int dv) {
  (void)B, (void)T, (void)Hk, (void)Hv, (void)dk, (void)dv;
  return 0;
}

sv_status gdn_chunk(const sv_states *states, const int32_t *slots, const sv_rows *q, const sv_rows *k,
                    const sv_rows *v, const float *g, const float *beta, const sv_rows *o, const int32_t *cu, int B,
                    int T, int Hk, int Hv, int dk, int dv, void *workspace, size_t ws_bytes, sv_stream_t stream) {
  (void)workspace, (void)ws_bytes;
  if (B < 0 || T < 0 || Hk < 1 || Hv < 1 || Hv % Hk != 0 || dk < 1 || dv < 1) return SV_ERR_INVALID_ARG;
  if (dk != 64 && dk != 128) return SV_ERR_UNSUPPORTED;
  if (Hv > 65535 || B > gdn::MAX_POOL_B || T > 0x40000000 || dv > 65536) return SV_ERR_UNSUPPORTED;
  if (sv_status e = gdn::check_states(states, Hv, dk, dv)) return e;
  for (const sv_rows *r : {q, k, v, o})
    if (!paged::good_rows(r, T)) return SV_ERR_INVALID_ARG;
  if (T > 0 && (!g || !beta || !paged::aligned(g, 4) || !paged::aligned(beta, 4))) return SV_ERR_INVALID_ARG;
  if (B > 0 && (!slots || !cu || !paged::aligned(slots, 4) || !paged::aligned(cu, 4))) return SV_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return SV_OK;
  gdn::PoolParams P{};
  P.states = *states;
  P.slots = slots;
  P.q = *q, P.k = *k, P.v = *v, P.o = *o, P.g = g, P.b = beta;
  P.cu = cu;
  P.err = device_error_word();
  if (!P.err) return SV_ERR_CUDA;
  P.B = B, P.T = T, P.Hk = Hk, P.Hv = Hv, P.dv = dv;
  P.commit = 1;
  gdn::ChunkParams CP{};
  CP.p = P;
  CP.blocks = (dv + gdn::ROWS - 1) / gdn::ROWS;
  CP.stall = launch_flags() & SV_LAUNCH_TEST_STALL_COPY ? 1 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dk == 64 ? gdn::run_chunks<64>(CP, s) : gdn::run_chunks<128>(CP, s);
}

}  // extern "C"
