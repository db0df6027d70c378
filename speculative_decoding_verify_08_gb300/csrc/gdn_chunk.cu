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
// of three products and the register work between them.  Hence two kernels:
//  * prepare_kernel does what no state enters, for all blocks side by side: keys and
//    queries to fp16, K K^T and Q K^T (once for the value heads of a key head, where there
//    are many), decays, T and P, laid out in the workspace the way the chain's copies take them.
//  * chain_kernel walks the blocks of one sequence, value head and 128 rows of the
//    state.  Everything is held transposed, a row of the state (and of U, O) per lane
//    of tensor memory: X = S K^T, R = b (v - e^G X), U = R T^T, S' = U~ K; each result is
//    read by the threads that hold its rows and written back over itself as the
//    next product's first operand.  Two threads share a row; S stays in their
//    registers, in fp32.  Four warps write the output meanwhile, one issues the
//    products, one the copies (up to three blocks ahead).
//    A block takes it 2.5 us, 0.7 of them products; the rest is their results' way through
//    registers, four times a block.
//  * both_kernel is the chains with the preparation of later blocks on the SMs that they leave.
//    Measured (48 heads of 128 x 128 over 16): one sequence of 8192 tokens 331 us, of 77 15.7; eleven of 1 to
//    3001 tokens 198, of which preparation takes 78.
//  * Products take fp16 operands and fp32 sums.  S, R, U and T are fp32 values held
//    as two fp16 parts (x = hi + lo, 2^-22 of x), so that a state stays an fp32 one; what
//    only an output sees (S and U there, and P) is one part, 2^-11 beside the
//    output's own 2^-8.  (bf16 parts would need three for that, half as many
//    products again.)
//  * fp16 reaches from 2^-24 to 2^16, so everything is scaled by powers of two, exactly:
//    a key to a largest element in [2^-4, 2^-3) (k = 2^e k': b' = 4^e b, v' = 2^-e v,
//    u' = 2^e u is the same rule), a query likewise, and each row of S, and of R and U, by
//    factors of a block of their own, from bounds of what they can reach: S by its largest
//    element before and sum |U~| |k'|; U by its own: with b |k|^2 <= 2 a token adds at most
//    |b' v'| |k'| to a row's norm, so that |u'| <= |b' v'| + b' |k'| (|S| + 64 |b' v'| |k'|).  Both stand
//    below 2^15, so that the parts are off by 2^-22 of themselves, or 2^-39 of that bound.
//  * The inverse: four 16 x 16 blocks by forward substitution in fp32, then joined twice
//    by -T22 (A21 T11), which is as stable as the substitution.  Its entries are at most 45 (b' |k'|^2 <= 2,
//    and no |k'| is over 23 times another); they are held T_GAIN times as large, which fp16 still reaches,
//    so that small ones (a token seen through many decays) are off by 2^-34 only: a state that decays by e^-6.4 in
//    a block keeps 2^-22 of itself, and 2^-16 without that.
//  * G is summed in two fp32 parts and so are its differences: a gate that closes
//    (g = -1000) leaves the decays behind it exact.
#include "gdn_pool.cuh"
#include "tcgen05.cuh"

namespace sv {
namespace attn {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // attn.cu
}
namespace gdn {
namespace {

constexpr int C = 64;        // tokens of a block
constexpr int ROWS = 128;    // rows of the state a CTA holds (TMEM lanes)
constexpr int AS = 68;       // row stride of the inverse's fp32 matrix
constexpr int MAX_KEPT = 128;  // sequences whose lengths and places a CTA looks at itself
constexpr float G_LEAST = -10000.f;  // e^g is 0 long before
constexpr float P_GAIN = 1024.f;     // P is taken so much larger: decays down to 2^-24 keep their bits
constexpr float T_GAIN = 512.f;      // and A and T

// A block's scalars for one value head.
struct Scalars {
  float bv[C], bx[C], en[C], os1[C], os2[C];  // of v and of X (negative) in R, of T_GAIN U in U~, of the output's two products
  float gc;                                   // decay over the block
  float bk[2];                                // largest b' |k'|, of the first and of the last tokens
  float pad[61];
};
constexpr int PART = C * 128;  // bytes of one part of T, and of P
constexpr int HEAD_BYTES = 3 * PART + (int)sizeof(Scalars);  // T (hi, lo), P, scalars
static_assert(sizeof(Scalars) == 1536 && HEAD_BYTES % 512 == 0, "copies");
template <int DK>
__host__ __device__ constexpr int key_bytes() { return C * DK * 2; }  // a block's keys (and queries) of one key head

struct ChunkParams {
  PoolParams p;
  uint8_t *keys, *heads;  // [blocks][Hk][2][key_bytes], [blocks][Hv][HEAD_BYTES]
  int split;              // prepare_kernel: a CTA a value head, not a key head
  int early;              // the chains may start beside it
  int first;              // only a sequence's first blocks are prepared before the chains start (0: all)
  unsigned *made;         // [blocks][Hv]: a later block prepared, beside the chains
  unsigned *before;       // [B + 1]: blocks of the sequences before one, and of all (more than MAX_KEPT sequences)
  int makers;             // CTAs that do
  int row_blocks;         // of ROWS rows a value head
  int stall;              // test aid: the first block never arrives
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
// Whether `ok` holds for all threads of the rows' warps, which all come by.
__device__ __forceinline__ bool all_rows(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.red.and.pred q, 5, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float pow2_inverse(float x) { return __int_as_float((254 << 23) - __float_as_int(x)); }  // of a power of two

// Blocks that the workspace has places for: as many as sequences without common rows can have.
__host__ __device__ inline long long places(int B, int T) { return (long long)T / C + B; }

// A sequence's blocks stand behind those of all sequences before it that are not left out.  Sequences that
// share rows (their offsets fall) may have more blocks than there are places: all are left out then.
__device__ __forceinline__ unsigned blocks_of(const PoolParams &P, int b) { return ((unsigned)rows_of(P, b, false).y + C - 1) / C; }
// Places of up to MAX_KEPT sequences, four a lane of the warp (128 sequences of 2^24 blocks stay within 32 bits).
struct Places {
  unsigned before[4], all;
  // (b: the same in all lanes)
  __device__ __forceinline__ int first(int b) const {
    const int x = b & 3;
    return (int)__shfl_sync(0xffffffffu, x == 0 ? before[0] : x == 1 ? before[1] : x == 2 ? before[2] : before[3], b >> 2);
  }
};
__device__ __forceinline__ Places places_of(const PoolParams &P, int lane) {
  Places p;
  unsigned n[4], x = 0;
#pragma unroll
  for (int y = 0; y < 4; ++y) x += n[y] = 4 * lane + y < P.B ? blocks_of(P, 4 * lane + y) : 0u;
  const unsigned mine = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  p.all = __shfl_sync(0xffffffffu, x, 31);
  p.before[0] = x - mine;
#pragma unroll
  for (int y = 1; y < 4; ++y) p.before[y] = p.before[y - 1] + n[y - 1];
  return p;
}
// Of more sequences: once a call, by one CTA.
__global__ void __launch_bounds__(1024) places_kernel(const __grid_constant__ ChunkParams CP) {
  const PoolParams &P = CP.p;
  __shared__ unsigned sums[32];
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait();
  const unsigned most = (unsigned)places(P.B, P.T) + 1;  // (below 2^25; sums stay at it)
  unsigned all = 0;
  for (int b0 = 0; b0 < P.B; b0 += 1024) {
    const unsigned n = b0 + tid < P.B ? blocks_of(P, b0 + tid) : 0u;
    unsigned x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = min(x + y, most);
    }
    __syncthreads();  // (sums of the sequences before have been read)
    if (lane == 31) sums[tid >> 5] = x;
    __syncthreads();
    unsigned front = 0, round = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < (tid >> 5)) front = min(front + sums[w], most);
      round = min(round + sums[w], most);
    }
    if (b0 + tid < P.B) CP.before[b0 + tid] = min(min(all + front, most) + x, most) - n;
    all = min(all + round, most);
  }
  if (tid == 0) CP.before[P.B] = all;
}

// x + y of two-part values, the first part the value rounded.
__device__ __forceinline__ float2 add_parts(float2 x, float2 y) {
  const float s = x.x + y.x, t = s - x.x;
  const float e = ((x.x - (s - t)) + (y.x - t)) + (x.y + y.y);
  const float h = s + e;
  return make_float2(h, e - (h - s));
}

// ------------------------------------------------------------------ prepare --
template <int DK>
struct PL {
  static constexpr int KQ = 0;                        // [DK/64][128 rows][128 B]: keys in rows 0..63, queries behind
  static constexpr int A = KQ;                        // then: fp32 [64][AS], inverted in place
  static constexpr int FIRST = 128 * DK * 2 > C * AS * 4 ? 128 * DK * 2 : (C * AS * 4 + 1023) / 1024 * 1024;
  static constexpr int GH = FIRST;                    // G in units of log 2, two parts [2][64]
  static constexpr int EX = GH + 2 * C * 4;           // exponents of the largest elements [128]
  static constexpr int BAR = EX + 128 * 4;
  static constexpr int BYTES = BAR + 64;
};

// Operands of a warp's 16 x 8 x 16 product out of fp32 matrices of row stride AS, in two parts.
template <int N>
struct Parts {
  uint32_t hi[N], lo[N];
};
__device__ __forceinline__ void left_operand(Parts<4> &p, const float *a, int lane) {
#pragma unroll
  for (int z = 0; z < 4; ++z)
    split2(*reinterpret_cast<const f2 *>(a + ((lane >> 2) + 8 * (z & 1)) * AS + 2 * (lane & 3) + 8 * (z >> 1)), p.hi[z], p.lo[z]);
}
__device__ __forceinline__ void right_operand(Parts<2> &p, const float *a, int lane) {
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const float *x = a + (2 * (lane & 3) + 8 * z) * AS + (lane >> 2);
    split2(pack2(x[0], x[AS]), p.hi[z], p.lo[z]);
  }
}
__device__ __forceinline__ void multiply(float (&d)[4], const Parts<4> &l, const Parts<2> &r) {
  mma_f16_16816(d, l.lo[0], l.lo[1], l.lo[2], l.lo[3], r.hi[0], r.hi[1]);
  mma_f16_16816(d, l.hi[0], l.hi[1], l.hi[2], l.hi[3], r.lo[0], r.lo[1]);
  mma_f16_16816(d, l.hi[0], l.hi[1], l.hi[2], l.hi[3], r.hi[0], r.hi[1]);
}
// A product of two matrices that are held T_GAIN times as large, as such a matrix.
__device__ __forceinline__ void put_tile(float *a, const float (&d)[4], bool minus, int lane) {
  float *x = a + (lane >> 2) * AS + 2 * (lane & 3);
  const float f = minus ? -1.f / T_GAIN : 1.f / T_GAIN;
  *reinterpret_cast<float2 *>(x) = make_float2(f * d[0], f * d[1]);
  *reinterpret_cast<float2 *>(x + 8 * AS) = make_float2(f * d[2], f * d[3]);
}

// Prepares rows r0..r0+m-1, block w of the workspace, for value heads e0..e1-1 of key head hk: 128
// threads (pt), `smem` and 64 columns of tensor memory of their own.
template <int DK>
__device__ __forceinline__ void prepare(const ChunkParams &CP, uint8_t *smem, uint32_t tb, uint64_t *done, uint32_t parity,
                                        int barrier, int pt, int hk, int e0, int e1, int w, long long r0,
                                        int m) {
  using Y = PL<DK>;
  const PoolParams &P = CP.p;
  float *A = reinterpret_cast<float *>(smem + Y::A);
  float *gh = reinterpret_cast<float *>(smem + Y::GH), *gl = gh + C;
  int *ex = reinterpret_cast<int *>(smem + Y::EX);
  const int pw = pt >> 5, lane = pt & 31, group = P.Hv / P.Hk;
  auto sync = [&]() { named_barrier(barrier, 128); };
  // ---- keys and queries to fp16: eight threads a row ----
  {
    constexpr int PR = DK / 64;  // 16-byte pieces a thread
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(P.k.ptr) + (long long)hk * P.k.head_stride;
    const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(P.q.ptr) + (long long)hk * P.q.head_stride;
    uint8_t *image = CP.keys + ((size_t)w * P.Hk + hk) * 2 * key_bytes<DK>();
    const int s8 = pt & 7, t0 = pt >> 3;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const __nv_bfloat16 *src = half ? qp : kp;
      const long long stride = half ? P.q.token_stride : P.k.token_stride;
      uint4 v[4][PR];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int t = t0 + 16 * y;
#pragma unroll
        for (int z = 0; z < PR; ++z)
          v[y][z] = t < m ? *reinterpret_cast<const uint4 *>(src + (r0 + t) * stride + (s8 + 8 * z) * 8) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int t = t0 + 16 * y;
        uint32_t mx = 0;
#pragma unroll
        for (int z = 0; z < PR; ++z)  // (of finite values the larger has the larger bits)
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[y][z].x & 0x7fff7fffu, v[y][z].y & 0x7fff7fffu),
                                     __vmaxu2(v[y][z].z & 0x7fff7fffu, v[y][z].w & 0x7fff7fffu)));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        // (2^(250 - E) and its inverse both have to be normal: beyond, queries are left larger, still within
        // fp16, and keys are zeros, as beta can only be 0 there)
        const int top = (int)(max(mx & 0xffffu, mx >> 16) >> 7), E = imin(top, 249);
        const float f = top > 249 && half == 0 ? 0.f : pow2_field(250 - E);
        const f2 f2x = pack2(f, f);
        auto two = [&](uint32_t x) {
          const float2 p = unpack2(mul2(pack2(bf16lo(x), bf16hi(x)), f2x));
          return pack_f16x2(p.x, p.y);
        };
#pragma unroll
        for (int z = 0; z < PR; ++z) {
          const uint4 d = make_uint4(two(v[y][z].x), two(v[y][z].y), two(v[y][z].z), two(v[y][z].w));
          *reinterpret_cast<uint4 *>(smem + Y::KQ + z * 128 * 128 + swz(half * C + t, s8)) = d;
          if (e0 == 0) *reinterpret_cast<uint4 *>(image + half * key_bytes<DK>() + z * C * 128 + swz(t, s8)) = d;
        }
        if (s8 == 0) ex[half * C + t] = E;
      }
    }
  }
  fence_proxy_async();
  tc::fence_before_sync();
  sync();
  tc::fence_after_sync();
  // ---- K K^T over Q K^T ----
  if (pw == 0 && tc::elect_one()) {
    const uint64_t da = tc::smem_desc_sw128(smem_u32(smem + Y::KQ), 16, 1024);
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      const uint64_t d = da + ((ks >> 2) * 128 * 128 + (ks & 3) * 32) / 16;
      tc::mma_bf16(tb, d, d, tc::idesc_f16_f32(128, C, false), ks > 0);
    }
    tc::commit(done);
  }
  __syncwarp();
  mbar_wait(done, parity, P.err);
  __syncwarp();
  tc::fence_after_sync();
  const bool isP = pw >= 2;
  const int i = (pw & 1) * 32 + lane;  // this thread's row of A, or of P
  const float e_i = pow2_field(ex[i] + 4);  // 2^e of its key
  for (int e = e0; e < e1; ++e) {
    const int h = hk * group + e;
    uint8_t *out = CP.heads + ((size_t)w * P.Hv + h) * HEAD_BYTES;
    float be = 0.f;
    if (i < m) be = P.b[(r0 + i) * P.Hv + h];
    sync();  // A and G of the head before (the products' operands) have been read
    if (pw == 0) {  // running sums of the gates, in units of log 2, two tokens a lane
      auto gate = [&](int t) {
        float g = t < m ? P.g[(r0 + t) * P.Hv + h] : 0.f;
        g = g < G_LEAST ? G_LEAST : g;
        // log2(e) in two parts
        const float x = g * 1.44269502f;
        return make_float2(x, fmaf(g, 1.44269502f, -x) + g * 1.92596303e-8f);
      };
      const float2 g0 = gate(2 * lane), g1 = gate(2 * lane + 1);
      const float2 pair = add_parts(g0, g1);
      float2 x = pair;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float2 y = make_float2(__shfl_up_sync(0xffffffffu, x.x, o), __shfl_up_sync(0xffffffffu, x.y, o));
        if (lane >= o) x = add_parts(x, y);
      }
      const float2 before = make_float2(__shfl_up_sync(0xffffffffu, x.x, 1), __shfl_up_sync(0xffffffffu, x.y, 1));
      const float2 x0 = lane > 0 ? add_parts(before, g0) : g0;
      *reinterpret_cast<float2 *>(gh + 2 * lane) = make_float2(x0.x, x.x);
      *reinterpret_cast<float2 *>(gl + 2 * lane) = make_float2(x0.y, x.y);
    }
    sync();
    Scalars *S = reinterpret_cast<Scalars *>(out + 3 * PART);
    const float hi_i = gh[i], lo_i = gl[i], ga = ex2_approx(hi_i + lo_i);
    if (!isP) {
      const float bs = be * e_i;
      S->bv[i] = bs;
      S->bx[i] = -(bs * e_i * ga);
      S->en[i] = ex2_approx((gh[C - 1] - hi_i) + (gl[C - 1] - lo_i)) * (1.f / T_GAIN);
    } else {
      const float os = pow2_field(ex[C + i] + 4);
      S->os1[i] = os * ga;
      S->os2[i] = os * (1.f / P_GAIN);
      if (i == C - 1) S->gc = ga;
    }
    // ---- A (rows of the first two warps) and P ----
    {
      const float rf = isP ? P_GAIN : be * e_i * e_i * T_GAIN;
      const f2 rowf = pack2(rf, rf), hi2 = pack2(hi_i, hi_i), lo2 = pack2(lo_i, lo_i), neg = pack2(-1.f, -1.f);
      const int last = isP ? i : i - 1;  // columns up to it count
#pragma unroll
      for (int c0 = 0; c0 < 2; ++c0) {
        const bool any = c0 == 0 || (pw & 1);  // columns 32.. of rows 0..31 are zero
        uint32_t raw[32];  // (from tensor memory for every head: kept, they cost two blocks an SM)
        tc::ld32(tb + c0 * 32 + ((uint32_t)(pw * 32) << 16), raw);
        tc::wait_ld();
        if (!isP && c0 == (pw & 1)) {  // |k'|^2 of this row's key stands on the diagonal
          float kk = 0.f;
#pragma unroll
          for (int x = 0; x < 32; ++x) kk = x == lane ? __uint_as_float(raw[x]) : kk;
          // (of values that are not negative the larger has the larger bits)
          const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(rf) * (1.f / T_GAIN) * sqrtf(kk)));
          if (lane == 0) S->bk[pw] = __uint_as_float(top);
        }
#pragma unroll
        for (int x = 0; x < 32; x += 8) {
          const int j = c0 * 32 + x;
          f2 y[4] = {0, 0, 0, 0};
          if (any) {
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const f2 hj = *reinterpret_cast<const f2 *>(gh + j + 2 * z), lj = *reinterpret_cast<const f2 *>(gl + j + 2 * z);
              const float2 d = unpack2(add2(fma2(hj, neg, hi2), fma2(lj, neg, lo2)));
              const f2 kk = pack2(__uint_as_float(raw[x + 2 * z]), __uint_as_float(raw[x + 2 * z + 1]));
              const float2 t = unpack2(mul2(mul2(kk, rowf), pack2(ex2_approx(d.x), ex2_approx(d.y))));
              y[z] = pack2(j + 2 * z <= last ? t.x : 0.f, j + 2 * z + 1 <= last ? t.y : 0.f);
            }
          }
          if (isP) {
            auto h2 = [](f2 v) {
              const float2 p = unpack2(v);
              return pack_f16x2(p.x, p.y);
            };
            *reinterpret_cast<uint4 *>(out + 2 * PART + swz(i, j >> 3)) = make_uint4(h2(y[0]), h2(y[1]), h2(y[2]), h2(y[3]));
          } else {
            *reinterpret_cast<ulonglong2 *>(A + i * AS + j) = make_ulonglong2(y[0], y[1]);
            *reinterpret_cast<ulonglong2 *>(A + i * AS + j + 4) = make_ulonglong2(y[2], y[3]);
          }
        }
      }
    }
    sync();
    // ---- T = (I + A)^-1 in place: a 16 x 16 block a warp, a column a lane ----
    {
      const int o = pw * 16;
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float s0 = r == lane ? T_GAIN : 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < r; j += 4) {
          const float4 a = *reinterpret_cast<const float4 *>(A + (o + r) * AS + o + j);
          s0 = fmaf(-a.x, x[j], s0);
          if (j + 1 < r) s1 = fmaf(-a.y, x[j + 1], s1);
          if (j + 2 < r) s0 = fmaf(-a.z, x[j + 2], s0);
          if (j + 3 < r) s1 = fmaf(-a.w, x[j + 3], s1);
        }
        x[r] = (s0 + s1) * (1.f / T_GAIN);
      }
      __syncwarp();
      if (lane < 16) {
#pragma unroll
        for (int r = 0; r < 16; ++r) A[(o + r) * AS + o + lane] = x[r] * T_GAIN;
      }
    }
    sync();
    // joined: T21 = -T22 (A21 T11), 16 rows and columns of two pairs, then 32 of one; the
    // products in two fp16 parts too (on the CUDA cores their operands' way through shared
    // memory took longer than all else here)
    {
      const int o = (pw >> 1) * 32, n0 = o + (pw & 1) * 8;  // pair, eight columns
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const float *left = A + (o + 16) * AS + o + 16 * pass, *right = A + (o + 16 * pass) * AS + n0;
        Parts<4> l;
        Parts<2> r;
        left_operand(l, left, lane);
        right_operand(r, right, lane);
        multiply(d, l, r);
        sync();
        put_tile(A + (o + 16) * AS + n0, d, pass, lane);
        sync();
      }
    }
    {
      const int m0 = 32 + (pw & 1) * 16, n0 = (pw >> 1) * 16;  // 16 rows, 16 columns
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 32 * pass; k < 32 * pass + 32; k += 16) {
          Parts<4> l;
          left_operand(l, A + m0 * AS + k, lane);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            Parts<2> r;
            right_operand(r, A + k * AS + n0 + 8 * z, lane);
            multiply(d[z], l, r);
          }
        }
        sync();
#pragma unroll
        for (int z = 0; z < 2; ++z) put_tile(A + m0 * AS + n0 + 8 * z, d[z], pass, lane);
        sync();
      }
    }
    // ---- T in two parts: pieces of eight, a row's eight pieces side by side ----
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = (pt >> 3) + 16 * x, p = pt & 7;
      const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(A + r * AS + p * 8), d = *reinterpret_cast<const ulonglong2 *>(A + r * AS + p * 8 + 4);
      uint4 th, tl;
      split2(a.x, th.x, tl.x);
      split2(a.y, th.y, tl.y);
      split2(d.x, th.z, tl.z);
      split2(d.y, th.w, tl.w);
      *reinterpret_cast<uint4 *>(out + swz(r, p)) = th;
      *reinterpret_cast<uint4 *>(out + PART + swz(r, p)) = tl;
    }
  }
}

template <int DK>
__global__ void __launch_bounds__(128, 6) prepare_kernel(const __grid_constant__ ChunkParams CP) {
  using Y = PL<DK>;
  const PoolParams &P = CP.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(P.err, ERR_TIMEOUT);
    return;
  }
  uint64_t *done = reinterpret_cast<uint64_t *>(smem + Y::BAR);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  const int pt = threadIdx.x;
  pdl_wait();
  // ---- the block: sequence and first row ----
  const int group = P.Hv / P.Hk, heads = CP.split ? P.Hv : P.Hk;
  int w = blockIdx.x / heads, b, c;  // (heads of the same tokens side by side)
  const int head = blockIdx.x - w * heads, hk = CP.split ? head / group : head;
  const int e0 = CP.split ? head - hk * group : 0, e1 = CP.split ? e0 + 1 : group;
  unsigned all;
  if (CP.first) {
    const unsigned flags = (unsigned)places(P.B, P.T) * P.Hv;
    for (unsigned x = blockIdx.x * 128 + pt; x < flags; x += gridDim.x * 128) CP.made[x] = 0;
    b = w / CP.first, c = w - b * CP.first;
    const Places at = places_of(P, pt & 31);
    w = at.first(b) + c, all = at.all;
  } else if (P.B <= MAX_KEPT) {
    const Places at = places_of(P, pt & 31);
    // the last sequence that begins at or before it: the last of a lane's four, of the last such lane
    int mine = -1, from = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (4 * (pt & 31) + y < P.B && (int)at.before[y] <= w) mine = 4 * (pt & 31) + y, from = (int)at.before[y];
    const int lane = 31 - __clz(__ballot_sync(0xffffffffu, mine >= 0));  // (the first sequence begins at 0)
    b = __shfl_sync(0xffffffffu, mine, lane), c = w - __shfl_sync(0xffffffffu, from, lane), all = at.all;
  } else {
    int lo = 0, hi = P.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (CP.before[mid] <= (unsigned)w) lo = mid; else hi = mid - 1;
    }
    b = lo, c = w - (int)CP.before[b], all = CP.before[P.B];
  }
  const int2 own = rows_of(P, b, false);
  if ((long long)c * C >= own.y || all > (unsigned)places(P.B, P.T)) return;
  if (pt == 0) {
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (pt < 32) {
    tc::tmem_alloc(tmem_slot, 64u);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // The chains may start: what ran before this kernel is over, and every block of it that is still to
  // finish has its place and its tensor memory.
  if (CP.early) pdl_launch_dependents();
  prepare<DK>(CP, smem, tb, done, 0, 0, pt, hk, e0, e1, w, own.x + (long long)c * C, imin(C, own.y - c * C));
  tc::fence_before_sync();
  __syncthreads();
  if (pt < 32) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, 64u);
  }
}

// -------------------------------------------------------------------- chain --
// Eight warps hold the rows of S, two threads a row; four write the output; one
// fetches, one issues the products.
constexpr int ROW_WARPS = 8, OUT_WARPS = 4, FETCH = ROW_WARPS + OUT_WARPS, ISSUE = FETCH + 1;
constexpr int CHAIN_THREADS = (ROW_WARPS + OUT_WARPS + 4) * 32, STAGES = 3;
// Blocks of a sequence that are prepared before the chains where later ones are beside them (8192 tokens 332 us
// with 8, 338 with 4), and how many of those a value head at a time (sooner there; 346 us with none, 339 with 8,
// 331 with 16, 32 or 64).
constexpr int FIRST = 8, SOON = 16;

template <int DK>
struct CL {
  static constexpr int K = 0, Q = key_bytes<DK>(), T = 2 * key_bytes<DK>(), P = T + 2 * PART, V = P + PART;
  static constexpr int S = V + C * ROWS * 2;            // scalars
  static constexpr int STAGE = S + 2048;                // (1024-byte aligned)
  static constexpr int SCALE = 1024;                    // [2][ROWS] bf16x2: what the rows' two outputs are multiplied by
  static constexpr int XCHG = SCALE + 2 * ROWS * 4;     // [2][2][ROWS]
  static constexpr int RING = XCHG + 4 * ROWS * 4;
  static constexpr int BYTES = RING + STAGES * STAGE;
  static_assert(RING % 1024 == 0 && STAGE % 1024 == 0 && BYTES <= 227 * 1024, "shared memory");
  // tensor memory: S in two parts; X, then R over it (16 columns a k-step: hi, lo), then U
  // in one part; U, then U~ over it; S'; S Q^T; P U
  static constexpr uint32_t SH = 0, SL = DK / 2, X = 128, U = 192, D = 256, O1 = 384, O2 = 448;
  static constexpr int STEPS = DK / 32;  // k-steps of S that are one thread's
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tensor_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// A block of rows of one head's state: (32 columns, row, column group, head, slot).
__device__ __forceinline__ void state_load(void *dst, const CUtensorMap *map, int row, int head, int slot, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(0), "r"(row), "r"(0), "r"(head), "r"(slot), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void state_store(const CUtensorMap *map, const void *src, int row, int head, int slot) {
  asm volatile("cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4, %5}], [%6];" ::"l"(map), "r"(0),
               "r"(row), "r"(0), "r"(head), "r"(slot), "r"(smem_u32(src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

// Whether another CTA's flag is up, sooner or later.
__device__ __forceinline__ bool wait_flag(const unsigned *flag, unsigned *err) {
  unsigned x;
  const long long t0 = clock64();
  while (true) {
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(flag) : "memory");
    if (x) return true;
    if (clock64() - t0 > WAIT_LIMIT_CYCLES) {
      atomicOr(err, ERR_TIMEOUT);
      return false;
    }
    __nanosleep(100);
  }
}

// Item `id` of the chains.  `beside`: other CTAs of the launch prepare the blocks meanwhile.
template <int DK>
__device__ __forceinline__ void chain(const CUtensorMap &mapV, const CUtensorMap &mapS, const ChunkParams &CP, uint8_t *smem, int id, bool beside) {
  using Y = CL<DK>;
  const PoolParams &P = CP.p;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem);     // [STAGES]
  uint64_t *empty = full + STAGES;                         // [STAGES]
  uint64_t *s_ready = empty + STAGES;                      // [2] first and second half of each thread's k-steps of S
  uint64_t *x_done = s_ready + 2, *r_ready = x_done + 1, *u_done = r_ready + 2, *ut_ready = u_done + 1;  // (r_ready [2], as s_ready)
  uint64_t *d_done = ut_ready + 1, *o_done = d_done + 1, *o_free = o_done + 1, *idle = o_free + 1;
  uint64_t *s_here = idle + 1, *s_read = s_here + 1;       // the state in the last stage, and read
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_read + 1);
  int *pick = reinterpret_cast<int *>(tmem_slot + 1);
  uint32_t *scale = reinterpret_cast<uint32_t *>(smem + Y::SCALE);
  uint8_t *ring = smem + Y::RING;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1 + (i == 0 ? CP.stall : 0));
      mbar_init(&empty[i], ROW_WARPS + OUT_WARPS + 1);
    }
    for (uint64_t *b : {s_ready, s_ready + 1, r_ready, r_ready + 1, ut_ready, s_read}) mbar_init(b, ROW_WARPS);
    mbar_init(o_free, OUT_WARPS);
    for (uint64_t *b : {x_done, u_done, d_done, o_done, idle, s_here}) mbar_init(b, 1);
    fence_barrier_init();
    *pick = 0;
  }
  if (warp == FETCH) {
    tc::tmem_alloc(tmem_slot, 512u);
    tc::tmem_relinquish();
  }
  // (what the sequences are and their states: from before the kernel that prepares, which has waited
  // for it before it let this one start)
  // ---- the item: longest sequences first ----
  const int per = P.Hv * CP.row_blocks;
  int b = id / per;
  const int rest = id - b * per, h = rest / CP.row_blocks, i0 = (rest - h * CP.row_blocks) * ROWS;
  if (P.B > 1 && P.B <= MAX_KEPT) {
    int *len = reinterpret_cast<int *>(smem + Y::XCHG);
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
  int w0 = 0;                   // place of its first block
  int n = (own.y + C - 1) / C;  // blocks
  if (P.B > 1) {
    unsigned all;
    if (P.B <= MAX_KEPT) {
      const Places at = places_of(P, lane);
      w0 = at.first(b), all = at.all;
    } else {
      w0 = (int)CP.before[b], all = CP.before[P.B];
    }
    if (all > (unsigned)places(P.B, P.T)) n = 0;
  }
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const int r = (warp & 3) * 32 + lane;  // row, of those that hold one
  bool ok = true;
  // After a wait that ran out a warp goes on without waiting, issuing or storing (what it
  // reads of tensor memory then has no meaning; loads under a condition cost registers).
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (ok) ok = spin_wait(bar, parity, P.err);
    ok = __all_sync(0xffffffffu, ok);
  };
  auto arrive = [&](uint64_t *bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto scalars = [&](int st) { return reinterpret_cast<const Scalars *>(ring + st * Y::STAGE + Y::S); };

  // 512 threads start with 128 registers each: 256 * 184 + 256 * 72 is the same total
  if (warp >= FETCH) {
    setmaxnreg_dec<72>();
    if (warp == FETCH) {
      // ---------------------------------------------------------- copies --
      if (lane == 0) {
        const int hk = h / (P.Hv / P.Hk);
        int c = 0;
        if (n > 0 && slot >= 0) {
          mbar_arrive_expect_tx(s_here, ROWS * DK * 4);
          state_load(ring + (STAGES - 1) * Y::STAGE, &mapS, i0, h, slot, s_here);
        }
        pdl_wait();  // for what has been prepared
        for (; c < n && ok; ++c) {
          const int st = c % STAGES;
          if (c >= STAGES) ok = mbar_wait(&empty[st], (c / STAGES - 1) & 1, P.err);
          if (c == STAGES - 1 && slot >= 0) ok = mbar_wait(s_read, 0, P.err);
          if (beside && ok && c >= CP.first) {
            const unsigned *made = CP.made + (size_t)(w0 + c) * P.Hv;  // (keys come with the first of their value heads)
            ok = wait_flag(made + hk * (P.Hv / P.Hk), P.err) && wait_flag(made + h, P.err);
            fence_proxy_async();  // what was stored there is read by copies
          }
          if (!ok) break;
          uint8_t *at = ring + st * Y::STAGE;
          mbar_arrive_expect_tx(&full[st], 2 * key_bytes<DK>() + HEAD_BYTES + C * ROWS * 2);
          const size_t place = (size_t)(w0 + c) * P.Hv + h;
          bulk_load(at + Y::K, CP.keys + ((size_t)(w0 + c) * P.Hk + hk) * 2 * key_bytes<DK>(), 2 * key_bytes<DK>(), &full[st]);
          bulk_load(at + Y::T, CP.heads + place * HEAD_BYTES, 3 * PART, &full[st]);
          bulk_load(at + Y::S, CP.heads + place * HEAD_BYTES + 3 * PART, sizeof(Scalars), &full[st]);
          tensor_load_3d(at + Y::V, &mapV, i0, h, own.x + c * C, &full[st]);
        }
        if (n > 0 && slot >= 0) mbar_wait(s_here, 0, P.err);  // no copy may outlive the CTA
        if (!ok)
          for (int k = imax(0, c - STAGES); k < c && mbar_wait(&full[k % STAGES], (k / STAGES) & 1, P.err); ++k) {
          }
      }
      __syncwarp();
    } else if (warp == ISSUE) {
      // -------------------------------------------------------- products --
      const bool leader = tc::elect_one();
      constexpr uint32_t IDN = tc::idesc_f16_f32(128, C, false), IDD = tc::idesc_f16_f32(128, DK, true);
      const uint64_t d_row = tc::smem_desc_sw128(smem_u32(ring), 16, 1024), d_col = tc::smem_desc_sw128(smem_u32(ring), C * 128, 1024);
      const uint32_t row_hi = (uint32_t)(d_row >> 32), col_hi = (uint32_t)(d_col >> 32);
      for (int c = 0; c < n; ++c) {
        const int st = c % STAGES;
        const uint32_t par = c & 1, lo = (uint32_t)d_row + st * (Y::STAGE / 16), lot = (uint32_t)d_col + st * (Y::STAGE / 16);
        wait(&full[st], (c / STAGES) & 1);
        // X = S K^T, as the parts of S come
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          wait(&s_ready[x], par);
          tc::fence_after_sync();
          if (leader && ok) {
#pragma unroll
            for (int y = 0; y < Y::STEPS; ++y) {
              const int ks = (y / (Y::STEPS / 2)) * Y::STEPS + x * (Y::STEPS / 2) + y % (Y::STEPS / 2);
#pragma unroll
              for (int p = 0; p < 2; ++p)
                tc::mma_bf16_ts(tb + Y::X, tb + (p ? Y::SL : Y::SH) + ks * 8, lo + (Y::K + (ks >> 2) * C * 128 + (ks & 3) * 32) / 16, row_hi,
                                IDN, x > 0 || y > 0 || p > 0);
            }
            if (x == 1) tc::commit(x_done);
          }
          __syncwarp();
        }
        // U = R T^T, the first 16 tokens of each thread, then the rest
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          wait(&r_ready[x], par);
          tc::fence_after_sync();
          if (leader && ok) {
#pragma unroll
            for (int ks = x; ks < C / 16; ks += 2)
#pragma unroll
              for (int p = 0; p < 3; ++p)  // hi hi, lo hi, hi lo
                tc::mma_bf16_ts(tb + Y::U, tb + Y::X + ks * 16 + (p == 1 ? 8 : 0), lo + (Y::T + (p == 2 ? PART : 0) + ks * 32) / 16, row_hi, IDN,
                                x > 0 || ks > 0 || p > 0);
            if (x == 1) tc::commit(u_done);
          }
          __syncwarp();
        }
        // S Q^T
        if (c > 0) wait(o_free, par ^ 1);
        tc::fence_after_sync();
        if (leader && ok) {
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            tc::mma_bf16_ts(tb + Y::O1, tb + Y::SH + ks * 8, lo + (Y::Q + (ks >> 2) * C * 128 + (ks & 3) * 32) / 16, row_hi, IDN, ks > 0);
        }
        __syncwarp();
        // S' = U~ K, then P U
        wait(ut_ready, par);
        tc::fence_after_sync();
        if (leader && ok) {
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
#pragma unroll
            for (int p = 0; p < 2; ++p)
              tc::mma_bf16_ts(tb + Y::D, tb + Y::U + ks * 16 + p * 8, lot + (Y::K + ks * 2048) / 16, col_hi, IDD, ks > 0 || p > 0);
          tc::commit(d_done);
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
            tc::mma_bf16_ts(tb + Y::O2, tb + Y::X + ks * 16, lo + (Y::P + ks * 32) / 16, row_hi, IDN, ks > 0);
          tc::commit(o_done);
          tc::commit(&empty[st]);
        }
        __syncwarp();
      }
      if (leader) {  // every product issued has completed before tensor memory is released
        tc::commit(idle);
        spin_wait(idle, 0, P.err);
      }
      __syncwarp();
    }
  } else if (warp >= ROW_WARPS) {
    // ---------------------------------------------------------- output --
    setmaxnreg_dec<72>();
    const long long step = P.o.token_stride;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(P.o.ptr) + own.x * step + (long long)h * P.o.head_stride + i0 + r;
    for (int c = 0; c < n; ++c) {
      const int st = c % STAGES;
      const Scalars *Z = scalars(st);
      // (o_done alone cannot run ahead of this warp; the rows' scale was written before the
      // products that it reports were let go)
      wait(o_done, c & 1);
      tc::fence_after_sync();
      const uint32_t scales = scale[(c & 1) * ROWS + r];
      const f2 f1 = pack2(bf16lo(scales), bf16lo(scales)), f2_ = pack2(bf16hi(scales), bf16hi(scales));
      const int some = i0 + r < P.dv && ok ? own.y - c * C : 0;
      // all of it is read before any is stored: the next block's products wait for it
      uint32_t y[C / 2];
#pragma unroll
      for (int t = 0; t < C; t += 8) {
        uint32_t a[8], d[8];
        tc::ld8(tb + Y::O1 + t + lane_off, a);
        tc::ld8(tb + Y::O2 + t + lane_off, d);
        tc::wait_ld();
#pragma unroll
        for (int z = 0; z < 8; z += 2) {
          const f2 s1 = *reinterpret_cast<const f2 *>(&Z->os1[t + z]), s2 = *reinterpret_cast<const f2 *>(&Z->os2[t + z]);
          const f2 x = fma2(pack2(__uint_as_float(a[z]), __uint_as_float(a[z + 1])), mul2(s1, f1),
                            mul2(pack2(__uint_as_float(d[z]), __uint_as_float(d[z + 1])), mul2(s2, f2_)));
          const float2 v = unpack2(x);
          y[(t + z) / 2] = pack_bf16x2(v.x, v.y);
        }
      }
      tc::fence_before_sync();
      arrive(o_free);
      if (some >= C) {
#pragma unroll
        for (int t = 0; t < C / 2; ++t) {
          *reinterpret_cast<uint16_t *>(out) = (uint16_t)y[t];
          *reinterpret_cast<uint16_t *>(out + step) = (uint16_t)(y[t] >> 16);
          out += 2 * step;
        }
      } else {  // the last block: nothing behind the sequence is written
#pragma unroll
        for (int t = 0; t < C / 2; ++t) {
          if (2 * t < some) *reinterpret_cast<uint16_t *>(out) = (uint16_t)y[t];
          if (2 * t + 1 < some) *reinterpret_cast<uint16_t *>(out + step) = (uint16_t)(y[t] >> 16);
          out += 2 * step;
        }
      }
      arrive(&empty[st]);
    }
  } else {
    // ------------------------------------------------------- rows of S --
    setmaxnreg_inc<184>();
    constexpr int SC = DK / 2;  // columns of S that are this thread's
    const int hf = warp >> 2;
    float *xchg = reinterpret_cast<float *>(smem + Y::XCHG);
    uint32_t trades = 0;
    // the larger of a value that both threads of a row have
    auto both = [&](float x) {
      float *at = xchg + (trades & 1) * 2 * ROWS + r;
      ++trades;
      at[hf * ROWS] = x;
      named_barrier(1 + (warp & 3), 64);
      return fmaxf(x, at[(hf ^ 1) * ROWS]);
    };
    // 16 bytes of this row's state in a stage (32 columns a group, pieces swizzled as the copies do)
    auto piece = [&](int stage, int e) {
      const int x = hf * SC / 4 + e;
      return reinterpret_cast<ulonglong2 *>(ring + stage * Y::STAGE + (x >> 3) * ROWS * 128 + r * 128 + (((x & 7) ^ (r & 7)) << 4));
    };
    const bool kept = slot >= 0 && n > 0;
    f2 S[SC / 2];
    float m = 0.f, sc = 1.f;
    if (kept) wait(s_here, 0);
#pragma unroll
    for (int e = 0; e < SC / 4; ++e) {  // (rows past the head's come as zeros)
      const ulonglong2 x = kept ? *piece(STAGES - 1, e) : make_ulonglong2(0, 0);
      S[2 * e] = x.x, S[2 * e + 1] = x.y;
      const float2 y = unpack2(x.x), z = unpack2(x.y);
      m = fmaxf(m, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(z.x), fabsf(z.y))));
    }
    if (kept) arrive(s_read);
    // scale of a row: 2^-k with at most 1 behind it
    auto scale_of = [&](float most) { return pow2_field(253 - imin(imax(__float_as_int(most) >> 23, 1), 250)); };
    // S (held scaled) as the next product's operand, a k-step at a time; the largest |S| of it
    auto put_state = [&]() {
      __half2 most = __float2half2_rn(0.f);
#pragma unroll
      for (int g = 0; g < Y::STEPS; ++g) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          split2(S[8 * g + e], hi[e], lo[e]);
          most = __hmax2(most, __habs2(*reinterpret_cast<__half2 *>(&hi[e])));
        }
        tc::st8(tb + Y::SH + hf * (SC / 2) + 8 * g + lane_off, hi);
        tc::st8(tb + Y::SL + hf * (SC / 2) + 8 * g + lane_off, lo);
        if ((g + 1) % (Y::STEPS / 2) == 0) {
          tc::wait_st();
          tc::fence_before_sync();
          arrive(&s_ready[g / (Y::STEPS / 2)]);
        }
      }
      return fmaxf(__low2float(most), __high2float(most));
    };
    if (n > 0) {
      sc = scale_of(both(m * 0x1p-15f));
      const f2 sc2 = pack2(sc, sc);
#pragma unroll
      for (int e = 0; e < SC / 2; ++e) S[e] = mul2(S[e], sc2);
      m = put_state();
    }
    // values of this thread's tokens, two a register, when they are there
    uint32_t vb[16];
    auto load_values = [&](int stage, uint32_t parity) {
      wait(&full[stage], parity);
      const uint16_t *v = reinterpret_cast<const uint16_t *>(ring + stage * Y::STAGE + Y::V) + hf * 32 * ROWS + r;
#pragma unroll
      for (int t = 0; t < 16; ++t) vb[t] = v[2 * t * ROWS] | (uint32_t)v[(2 * t + 1) * ROWS] << 16;
    };
    int st = 0;
    uint32_t phase = 0;
    if (n > 0) load_values(0, 0);
    for (int c = 0; c < n; ++c) {
      const uint32_t par = c & 1;
      const Scalars *Z = scalars(st);
      float scr;  // the scale of R, U and what comes of them
      // R = b (v - e^G X), a k-step (16 tokens) at a time
      {
        const int some = own.y - c * C - hf * 32;
        f2 w[16];  // b' v' of two tokens each, zeros past the sequence's end
        float wm = 0.f;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          uint32_t x = vb[t] << 16, y = vb[t] & 0xffff0000u;
          if (some < 32) x = 2 * t < some ? x : 0u, y = 2 * t + 1 < some ? y : 0u;
          w[t] = mul2(pack2(__uint_as_float(x), __uint_as_float(y)), *reinterpret_cast<const f2 *>(&Z->bv[hf * 32 + 2 * t]));
          const float2 z = unpack2(w[t]);
          wm = fmaxf(wm, fmaxf(fabsf(z.x), fabsf(z.y)));
        }
        // what U can reach, twice as the two halves of a row have terms of their own; and not so little beside
        // the state that the step from its scale to this one leaves fp32 (nothing at all where beta is 0)
        const float bk = fmaxf(Z->bk[0], Z->bk[1]), isc = pow2_inverse(sc), wl = wm * 0x1p-14f;
        scr = scale_of(both(fmaf(bk, 12.f * m * (isc * 0x1p-14f) + 91.f * wl, wl) + isc * 0x1p-94f));
        if (hf == 0) scale[par * ROWS + r] = pack_bf16x2(isc, pow2_inverse(scr));  // (powers of two)
        const f2 scr2 = pack2(scr, scr);
#pragma unroll
        for (int t = 0; t < 16; ++t) w[t] = mul2(w[t], scr2);
        const float rise = scr * isc;
        const f2 rise2 = pack2(rise, rise);
        wait(x_done, par);
        tc::fence_after_sync();
        uint32_t raw2[2][16];
        tc::ld16(tb + Y::X + hf * 32 + lane_off, raw2[0]);
        tc::ld16(tb + Y::X + hf * 32 + 16 + lane_off, raw2[1]);
        tc::wait_ld();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t hi[8], lo[8];
          const uint32_t (&raw)[16] = raw2[g];
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const int at = hf * 32 + 16 * g + 2 * t;
            const f2 bx = mul2(*reinterpret_cast<const f2 *>(&Z->bx[at]), rise2);
            split2(fma2(bx, pack2(__uint_as_float(raw[2 * t]), __uint_as_float(raw[2 * t + 1])), w[8 * g + t]), hi[t], lo[t]);
          }
          tc::st8(tb + Y::X + hf * 32 + 16 * g + lane_off, hi);
          tc::st8(tb + Y::X + hf * 32 + 16 * g + 8 + lane_off, lo);
          tc::wait_st();
          tc::fence_before_sync();
          arrive(&r_ready[g]);
        }
      }
      __half2 um = __float2half2_rn(0.f);
      {
        wait(u_done, par);
        tc::fence_after_sync();
        uint32_t raw2[2][16];
        tc::ld16(tb + Y::U + hf * 32 + lane_off, raw2[0]);
        tc::ld16(tb + Y::U + hf * 32 + 16 + lane_off, raw2[1]);
        tc::wait_ld();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t hi[8], lo[8], u[8];
          const uint32_t (&raw)[16] = raw2[g];
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const f2 ad = pack2(__uint_as_float(raw[2 * t]), __uint_as_float(raw[2 * t + 1]));
            const float2 one = unpack2(mul2(ad, pack2(1.f / T_GAIN, 1.f / T_GAIN)));
            u[t] = pack_f16x2(one.x, one.y);
            split2(mul2(ad, *reinterpret_cast<const f2 *>(&Z->en[hf * 32 + 16 * g + 2 * t])), hi[t], lo[t]);
            um = __hmax2(um, __habs2(*reinterpret_cast<__half2 *>(&hi[t])));
          }
          tc::st8(tb + Y::U + hf * 32 + 16 * g + lane_off, hi);
          tc::st8(tb + Y::U + hf * 32 + 16 * g + 8 + lane_off, lo);
          tc::st8(tb + Y::X + hf * 32 + 16 * g + lane_off, u);
        }
        tc::wait_st();
        tc::fence_before_sync();
        arrive(ut_ready);
      }
      const float gc = Z->gc;
      arrive(&empty[st]);
      st = st + 1 == STAGES ? 0 : st + 1;
      phase ^= st == 0;
      const float isc = pow2_inverse(sc), iscr = pow2_inverse(scr);
      // elements of k' are below 2^-3, 64 tokens: |S'| <= 8 |U~|; twice, as above (behind the last block too,
      // where what was added may be far larger than the state was)
      const float next = scale_of(both(gc * m * (isc * 0x1p-14f) + 8.f * fmaxf(__low2float(um), __high2float(um)) * (iscr * 0x1p-14f)));
      if (c + 1 < n) load_values(st, phase);
      // Parts end at 2^-25.  Where a row shows anything of S, the step to the new scale is below 2^38, and where it
      // does not, a larger step finds S below 2^-40 of its bound: it counts as 0.  Likewise an update that
      // shows nothing is 0, whatever multiplies it.
      const float step = next * isc, keep_all = step <= 0x1p126f ? gc * step : gc * isc * next;  // (a large one: gc is small)
      const float keep = keep_all <= 0x1p40f ? keep_all : 0.f, add = fminf(next * iscr, 0x1p126f);
      sc = next;
      const f2 keep2 = pack2(keep, keep), add_2 = pack2(add, add);
#pragma unroll
      for (int e = 0; e < SC / 2; ++e) S[e] = mul2(S[e], keep2);
      wait(d_done, par);
      tc::fence_after_sync();
      uint32_t raw[SC / 16][16];
#pragma unroll
      for (int g = 0; g < SC / 16; ++g) tc::ld16(tb + Y::D + hf * SC + 16 * g + lane_off, raw[g]);
      tc::wait_ld();
#pragma unroll
      for (int g = 0; g < SC / 16; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          S[8 * g + e] = fma2(pack2(__uint_as_float(raw[g][2 * e]), __uint_as_float(raw[g][2 * e + 1])), add_2, S[8 * g + e]);
      if (c + 1 < n) m = put_state();
    }
    if (kept) {
      // through the stage behind the last block's: nothing reads it any more
      const f2 isc2 = pack2(pow2_inverse(sc), pow2_inverse(sc));
      const int stage = n % STAGES;
#pragma unroll
      for (int e = 0; e < SC / 4; ++e) *piece(stage, e) = make_ulonglong2(mul2(S[2 * e], isc2), mul2(S[2 * e + 1], isc2));
      fence_proxy_async();
      // (all of the rows' warps are there, whatever ran out; nothing is stored if anything did)
      const bool all = all_rows(ok);
      if (all && tid == 0) state_store(&mapS, ring + stage * Y::STAGE, i0, h, slot);
      __syncwarp();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == FETCH) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, 512u);
  }
}

template <int DK>
__global__ void __launch_bounds__(CHAIN_THREADS, 1)
    chain_kernel(const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapS, const __grid_constant__ ChunkParams CP) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // swizzled tiles need it; so it is in a kernel without static shared memory
    if (threadIdx.x == 0) atomicOr(CP.p.err, ERR_TIMEOUT);
    return;
  }
  chain<DK>(mapV, mapS, CP, smem, blockIdx.x, false);
}

// The chains, and the preparation of all but a sequence's first blocks beside them: few
// items (one sequence: a chain a value head) leave most SMs idle.  The launch's first CTAs prepare, block
// by block in the order in which the chains take them, and put up a flag for each; the chains
// wait for the flags.  The preparing CTAs wait for nobody and start first, so every wait ends.
constexpr int MAKER_GROUPS = CHAIN_THREADS / 128;
template <int DK>
__global__ void __launch_bounds__(CHAIN_THREADS, 1)
    both_kernel(const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapS, const __grid_constant__ ChunkParams CP) {
  using Y = PL<DK>;
  constexpr int OWN = (Y::BYTES + 1023) / 1024 * 1024;
  static_assert(MAKER_GROUPS * OWN <= CL<DK>::BYTES && MAKER_GROUPS * 64 <= 512, "a group's shared and tensor memory");
  const PoolParams &P = CP.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(P.err, ERR_TIMEOUT);
    return;
  }
  if ((int)blockIdx.x >= CP.makers) {
    chain<DK>(mapV, mapS, CP, smem, blockIdx.x - CP.makers, true);
    return;
  }
  const int g = threadIdx.x >> 7, pt = threadIdx.x & 127;
  uint8_t *own = smem + g * OWN;
  uint64_t *done = reinterpret_cast<uint64_t *>(own + Y::BAR);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Y::BAR + 8);
  if (pt == 0) {
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (threadIdx.x < 32) {
    tc::tmem_alloc(tmem_slot, MAKER_GROUPS * 64u);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();
  const int group = P.Hv / P.Hk;
  const Places at = places_of(P, threadIdx.x & 31);  // (few items, so few sequences)
  int most = 0;  // blocks of the longest sequence
  for (int b = threadIdx.x & 31; b < P.B; b += 32) most = imax(most, (rows_of(P, b, false).y + C - 1) / C);
  most = at.all > (unsigned)places(P.B, P.T) ? 0 : __reduce_max_sync(0xffffffffu, most);
  // the next blocks a value head at a time, those behind them a key head
  const int later = imax(0, most - CP.first), soon = imin(later, SOON);
  const long long single = (long long)soon * P.B * P.Hv, tasks = single + (long long)(later - soon) * P.B * P.Hk;
  uint32_t parity = 0;
  for (long long x = blockIdx.x + (long long)g * CP.makers; x < tasks; x += (long long)MAKER_GROUPS * CP.makers) {
    const bool one = x < single;
    const long long z = one ? x : x - single;
    const int heads = one ? P.Hv : P.Hk;
    const long long y = z / heads;
    const int head = (int)(z - y * heads), n = (int)(y / P.B), b = (int)(y - (long long)n * P.B);
    const int c = CP.first + (one ? n : soon + n), hk = one ? head / group : head;
    const int e0 = one ? head - hk * group : 0, e1 = one ? e0 + 1 : group;
    const int2 rows = rows_of(P, b, false);
    if (c * C >= rows.y) continue;
    const int w = at.first(b) + c;
    prepare<DK>(CP, own, tb + 64 * g, done, parity, 1 + g, pt, hk, e0, e1, w, rows.x + (long long)c * C, imin(C, rows.y - c * C));
    parity ^= 1;
    __threadfence();
    fence_proxy_async();
    named_barrier(1 + g, 128);
    for (int e = e0 + pt; e < e1; e += 128)
      asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(&CP.made[(size_t)w * P.Hv + hk * group + e]), "r"(1u) : "memory");
  }
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x < 32) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, MAKER_GROUPS * 64u);
  }
}

inline size_t padded(int dv) { return ((size_t)dv + ROWS - 1) / ROWS * ROWS; }

template <int DK>
sv_status run_chunks(ChunkParams &CP, cudaStream_t s) {
  const PoolParams &P = CP.p;
  const long long items = (long long)P.B * P.Hv * CP.row_blocks, blocks = places(P.B, P.T);  // (checked: 31 bits)
  // values (column, head, token) in boxes of 128 x 1 x 64, zeros past the last column
  auto fn = attn::encode_fn();
  if (!fn) return SV_ERR_CUDA;
  CUtensorMap mv;
  // the stride of a dimension of one is never used, but has to be a valid one
  cuuint64_t dims[3] = {(cuuint64_t)P.dv, (cuuint64_t)P.Hv, (cuuint64_t)P.T};
  cuuint64_t strides[2] = {P.Hv > 1 ? (cuuint64_t)P.v.head_stride * 2 : 16, P.T > 1 ? (cuuint64_t)P.v.token_stride * 2 : 16};
  cuuint32_t box[3] = {ROWS, 1, C}, estr[3] = {1, 1, 1};
  if (fn(&mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, P.v.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return SV_ERR_CUDA;
  // states (32 columns, row of the head, column group, head, slot) in boxes of 32 x 128 x all, 128-byte
  // swizzle: rows past the head's are read as zeros and not written
  CUtensorMap ms;
  cuuint64_t sdims[5] = {32, (cuuint64_t)P.dv, DK / 32, (cuuint64_t)P.Hv, (cuuint64_t)P.states.num_slots};
  cuuint64_t sstr[4] = {DK * 4, 128, (cuuint64_t)P.dv * DK * 4,
                        P.states.num_slots > 1 ? (cuuint64_t)P.states.slot_stride * 4 : 16};
  cuuint32_t sbox[5] = {32, ROWS, DK / 32, 1, 1}, sest[5] = {1, 1, 1, 1, 1};
  if (fn(&ms, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 5, P.states.ptr, sdims, sstr, sbox, sest, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return SV_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return SV_ERR_CUDA;
  // Few items: all but the first blocks are prepared while the chains run (one sequence of 8192
  // tokens, 48 heads of 128 x 128: 332 us against 392; 2000 tokens 103 against 110; 1000 would be 61 against 64).
  CP.first = items <= sms / 2 && P.B <= MAX_KEPT && P.T > 2LL * FIRST * C * P.B ? FIRST : 0;
  const long long before = CP.first ? (long long)P.B * FIRST : blocks;
  // A value head a CTA while all of them are on the SMs at once, its key head's products made anew for
  // each (77 tokens: 15.6 us against 21.8; but eleven prompts of 1 to 3001 tokens 225 us against 198).
  CP.split = before * P.Hv <= 6LL * sms;
  const long long grid = before * (CP.split ? P.Hv : P.Hk);
  // Chains that find SMs of their own fetch their states meanwhile (77 tokens 15.6 us against 17.1); others would
  // only take places early (eleven prompts 211 us against 198).
  CP.early = !CP.first && grid + items <= sms;
  if (P.B > MAX_KEPT && launch_early(places_kernel, dim3(1), dim3(1024), 0, s, CP) != cudaSuccess) return SV_ERR_CUDA;
  cudaError_t e = launch_early(prepare_kernel<DK>, dim3((unsigned)grid), dim3(128), (size_t)PL<DK>::BYTES, s, CP);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  const size_t smem = CL<DK>::BYTES;
  if (!CP.first) return from_cuda(launch_early(chain_kernel<DK>, dim3((unsigned)items), dim3(CHAIN_THREADS), smem, s, mv, ms, CP));
  // Three to two chains keep up with them, and more slow the chains down: 8192 tokens, 48 chains, 332 us
  // with 72, 334 with 88, 351 with 104, 342 with 60, 360 with 40; 32 chains 328 with 48 to 96, 347 with 120, 344 with
  // 32.  Beside few chains as many as leave each SM pair one CTA (8 chains 320 to 323 with any from 16 to 140, 2 chains
  // 314 to 317).
  CP.makers = imin(sms - (int)items, imax(3 * (int)items / 2, sms / 2 - (int)items));
  return from_cuda(launch_early(both_kernel<DK>, dim3((unsigned)(CP.makers + items)), dim3(CHAIN_THREADS), smem, s, mv, ms, CP));
}

}  // namespace
}  // namespace gdn
}  // namespace sv

using namespace sv;

extern "C" {

size_t gdn_chunk_workspace_bytes(int B, int T, int Hk, int Hv, int dk, int dv) {
  if (B < 1 || T < 1 || Hk < 1 || Hv < 1 || dv < 1 || (dk != 64 && dk != 128)) return 0;
  const size_t per = (size_t)Hk * 4 * gdn::C * dk + (size_t)Hv * (gdn::HEAD_BYTES + 4);
  return (size_t)gdn::places(B, T) * per + ((size_t)B + 1) * 4;
}

sv_status gdn_chunk(const sv_states *states, const int32_t *slots, const sv_rows *q, const sv_rows *k,
                    const sv_rows *v, const float *g, const float *beta, const sv_rows *o, const int32_t *cu, int B,
                    int T, int Hk, int Hv, int dk, int dv, void *workspace, size_t ws_bytes, sv_stream_t stream) {
  if (B < 0 || T < 0 || Hk < 1 || Hv < 1 || Hv % Hk != 0 || dk < 1 || dv < 1) return SV_ERR_INVALID_ARG;
  if (dk != 64 && dk != 128) return SV_ERR_UNSUPPORTED;
  if (Hv > 65535 || B > gdn::MAX_POOL_B || T > 0x40000000 || dv > 65536) return SV_ERR_UNSUPPORTED;
  if (sv_status e = gdn::check_states(states, Hv, dk, dv)) return e;
  if (states->slot_stride > ((int64_t)1 << 37)) return SV_ERR_UNSUPPORTED;  // (a tensor map's bound is 2^40 bytes)
  for (const sv_rows *r : {q, k, v, o})
    if (!paged::good_rows(r, T)) return SV_ERR_INVALID_ARG;
  if (T > 0 && (!g || !beta || !paged::aligned(g, 4) || !paged::aligned(beta, 4))) return SV_ERR_INVALID_ARG;
  if (B > 0 && (!slots || !cu || !paged::aligned(slots, 4) || !paged::aligned(cu, 4))) return SV_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return SV_OK;
  // a tensor map steps by every stride: values that repeat (stride 0) have none
  if ((T > 1 && !v->token_stride) || (Hv > 1 && !v->head_stride)) return SV_ERR_UNSUPPORTED;
  const int row_blocks = (int)(gdn::padded(dv) / gdn::ROWS);
  if ((long long)B * Hv * row_blocks > 0x7fffffffLL || gdn::places(B, T) * Hv > 0x7fffffffLL) return SV_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < gdn_chunk_workspace_bytes(B, T, Hk, Hv, dk, dv)) return SV_ERR_WORKSPACE;
  if (!paged::aligned(workspace, 16)) return SV_ERR_INVALID_ARG;
  gdn::ChunkParams CP{};
  gdn::PoolParams &P = CP.p;
  P.states = *states;
  P.slots = slots;
  P.q = *q, P.k = *k, P.v = *v, P.o = *o, P.g = g, P.b = beta;
  P.cu = cu;
  P.err = device_error_word();
  if (!P.err) return SV_ERR_CUDA;
  P.B = B, P.T = T, P.Hk = Hk, P.Hv = Hv, P.dv = dv;
  P.commit = 1;
  CP.keys = static_cast<uint8_t *>(workspace);
  CP.heads = CP.keys + (size_t)gdn::places(B, T) * Hk * 4 * gdn::C * dk;
  CP.made = reinterpret_cast<unsigned *>(CP.heads + (size_t)gdn::places(B, T) * Hv * gdn::HEAD_BYTES);
  CP.before = CP.made + (size_t)gdn::places(B, T) * Hv;
  CP.row_blocks = row_blocks;
  CP.stall = launch_flags() & SV_LAUNCH_TEST_STALL_COPY ? 1 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // A block costs as much with one token as with 64; token by token is faster up to some eight tokens a
  // sequence (48 heads of 128 x 128: one sequence of 16 tokens 12 us against 13, of 24 17 against 13;
  // two of 8 10 against 16, of 12 19 against 16; eight of 8 26 against 40, of 12 35 against 40; 64 of 8 168
  // against 222, of 12 231 against 225).  The rule is the whole call's: a long sequence among many short ones
  // takes 0.55 us a token, and short ones beside a long one a block each.
  if (T <= 16 || T <= 8LL * B) return gdn::launch_tokens(P, dk, s);
  return dk == 64 ? gdn::run_chunks<64>(CP, s) : gdn::run_chunks<128>(CP, s);
}

}  // extern "C"
