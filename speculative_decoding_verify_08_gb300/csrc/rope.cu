// rope.cu -- per-head RMS norm and position rotation of query and key rows,
// and their (and the values') way into a paged cache, in one pass.
//
// Row x of D elements of one (token, head):
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset)
//   (u, v) <- (u cos a - v sin a, u sin a + v cos a),  a = position * inv_freq[pair]
// computed in fp32 and rounded once.
//
// What bounds it: every row is read once and written once, so HBM at many
// tokens (if the instructions per byte stay few) and the launch at few.  Hence:
//  * A thread keeps one head and takes it at N consecutive tokens: the head's
//    kind, weights and strides are worked out once, and the N rows' loads are
//    all in flight before anything is computed.  A block holds neighbouring
//    heads, so its loads of a token are one run of memory.  (Resident blocks
//    that walk over the tokens with the next rows' loads under way measured
//    94 us against 58 at 16381 tokens of 40 heads of 128: their own steps are
//    longer than the loads they hide.)
//  * D/(2V) lanes share a row.  A lane of a half-split rotation holds V elements of
//    the first half and their V partners of the second, so that a pair never
//    leaves its lane; V = 8 (16-byte accesses) unless rot_dim is no multiple
//    of 16 (V = 4).
//  * The sines of a block's tokens are made once, in shared memory, while the
//    rows' loads are in flight, and serve all its heads.
//  * Products and sums run two to an instruction (f32x2).
//  * The angle is an integer: position times a 64-bit fraction of a turn wraps
//    at whole turns by itself, so a far position loses nothing and no 64-bit
//    floating-point arithmetic is needed.
// Measured: 16381 tokens of 32 + 8 heads of 128: 57 us, 5.9 TB/s of 6.7; 30011
// tokens' keys and values of 4 heads of 256 into e4m3 pages: 38 us, 4.9 TB/s, held
// back by instructions (60% of the issue slots), into bf16 pages: 41 us, 6.0 TB/s; 4
// to 61 tokens: 2.3-2.5 us.
#include <cuda_fp8.h>

#include <cmath>

#include "paged.cuh"

namespace sv {
namespace rope {

constexpr int MAX_THREADS = 256;

enum Kind { TO_ROWS = 0, TO_BF16_PAGES = 1, TO_E4M3_PAGES = 2 };

struct Rows {
  char *p;
  long long ts, hs;  // element strides
};

struct Params {
  Rows q, k, v, qo, ko;
  const __nv_bfloat16 *qw, *kw;  // null: no norm
  float eps, offset;
  const unsigned long long *phases;  // null: no rotation
  const int *positions;
  int rot, split;  // rotated elements (0: none); pairs half a rotation apart
  const long long *slots;
  char *kc, *vc;
  const float *ks, *vs;
  long long page_stride, slot_stride, head_stride, num_slots;
  int page_size;
  int T, Hq, Hkv, H;  // H: rows per token (queries, keys, values)
  int gh;             // heads per block
  unsigned *err;
};

// Cosine and sine of position * phase / 2^64 turns.  The product's upper 32
// bits, as a signed fraction of a turn, are short by 2^-32 turns at most (and
// the phase's own rounding, 2^-34 at position 2^31), below the fp32 rounding of
// the fraction itself (2^-26).
__device__ __forceinline__ float2 turn(int pos, unsigned long long phase) {
  const unsigned long long f = (unsigned long long)(long long)pos * phase;
  float s, c;
  sincospif((float)(int)(f >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ f2 bf2(uint32_t v) { return pack2(bf16lo(v), bf16hi(v)); }
__device__ __forceinline__ uint32_t bf16x2(f2 v) {
  const float2 x = unpack2(v);
  return pack_bf16x2(x.x, x.y);
}
__device__ __forceinline__ uint32_t e4m3x4(f2 a, f2 b) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(unpack2(a), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(unpack2(b), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// V consecutive elements: loads, conversion to V/2 pairs, stores.
template <int V>
struct Group;
template <>
struct Group<8> {
  using type = uint4;
  static __device__ __forceinline__ void unpack(f2 (&y)[4], uint4 v) {
    y[0] = bf2(v.x), y[1] = bf2(v.y), y[2] = bf2(v.z), y[3] = bf2(v.w);
  }
  static __device__ __forceinline__ void store_bf16(char *p, const f2 (&y)[4]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(bf16x2(y[0]), bf16x2(y[1]), bf16x2(y[2]), bf16x2(y[3]));
  }
  static __device__ __forceinline__ void store_e4m3(char *p, const f2 (&y)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(e4m3x4(y[0], y[1]), e4m3x4(y[2], y[3]));
  }
};
template <>
struct Group<4> {
  using type = uint2;
  static __device__ __forceinline__ void unpack(f2 (&y)[2], uint2 v) { y[0] = bf2(v.x), y[1] = bf2(v.y); }
  static __device__ __forceinline__ void store_bf16(char *p, const f2 (&y)[2]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2(y[0]), bf16x2(y[1]));
  }
  static __device__ __forceinline__ void store_e4m3(char *p, const f2 (&y)[2]) {
    *reinterpret_cast<uint32_t *>(p) = e4m3x4(y[0], y[1]);
  }
};

template <int D, int KIND, int V, int N>
__global__ void __launch_bounds__(MAX_THREADS, N == 4 ? 3 : 4) rope_kernel(const Params P) {
  using GV = Group<V>;
  using G = typename GV::type;
  constexpr int LPR = D / (2 * V);  // lanes per row
  constexpr int H2 = V / 2;         // pairs of elements in a group
  // [N][V/2][rot/(2V)]: (cos, cos, sin, sin) of the pairs 2e and 2e+1 of every
  // lane side by side, so that the lanes' reads fall on all banks
  extern __shared__ __align__(16) float4 cs[];
  __shared__ long long dst[N];  // element of the token's slot, or -1
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid % LPR, grp = tid / LPR;
  const int head = blockIdx.y * P.gh + grp;
  const bool active = grp < P.gh && head < P.H;
  const int tok0 = blockIdx.x * N;
  const bool isq = head < P.Hq, isv = head >= P.Hq + P.Hkv;
  const int h = isq ? head : isv ? head - P.Hq - P.Hkv : head - P.Hq;
  const int half = P.rot / 2, rlanes = half / V;  // pairs; lanes that rotate
  const bool rotates = lane < rlanes;
  // first elements of this lane's two groups of V
  const int off0 = (P.split && rotates) ? V * lane : 2 * V * lane;
  const int off1 = (P.split && rotates) ? half + V * lane : 2 * V * lane + V;

  // what the angles and destinations need is asked for before the rows
  auto token_of = [&](int i) {
    int t = 0;
#pragma unroll
    for (int k = 1; k < N; ++k) t += i >= k * half ? 1 : 0;
    return t;
  };
  const int last = P.T - 1;
  unsigned long long phase = 0;
  long long slot = -1;
  int pos = 0;
  if (tid < N * half) {
    const int t = token_of(tid);
    phase = P.phases[tid - t * half];
    pos = P.positions[imin(tok0 + t, last)];
  }
  if (KIND != TO_ROWS && tid < N) slot = P.slots[imin(tok0 + tid, last)];
  G a[N], b[N];
  {
    const Rows src = isq ? P.q : isv ? P.v : P.k;
    const char *x = src.p + 2 * ((long long)tok0 * src.ts + (long long)h * src.hs);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = b[i] = G{};
      if (active && tok0 + i < P.T) {
        a[i] = *reinterpret_cast<const G *>(x + 2 * off0);
        b[i] = *reinterpret_cast<const G *>(x + 2 * off1);
      }
      x += 2 * src.ts;
    }
  }
  const __nv_bfloat16 *weight = isv ? nullptr : isq ? P.qw : P.kw;
  G wa{}, wb{};
  if (active && weight) {
    wa = *reinterpret_cast<const G *>(weight + off0);
    wb = *reinterpret_cast<const G *>(weight + off1);
  }
  const bool to_pages = KIND != TO_ROWS && !isq;
  float inv = 1.f;
  if (KIND == TO_E4M3_PAGES && active && to_pages) {
    const float *sp = isv ? P.vs : P.ks;
    if (sp) inv = 1.f / sp[h];
  }

  for (int i = tid; i < N * half; i += blockDim.x) {
    const int t = token_of(i), p = i - t * half, e = p % V;
    if (i != tid) {
      phase = P.phases[p];
      pos = P.positions[imin(tok0 + t, last)];
    }
    const float2 c = turn(pos, phase);
    float *at = reinterpret_cast<float *>(cs + (t * H2 + (e >> 1)) * rlanes + p / V) + (e & 1);
    at[0] = c.x;
    at[2] = c.y;
  }
  if (KIND != TO_ROWS && tid < N) {
    long long e = -1;
    if (slot >= P.num_slots) {
      atomicOr(P.err, ERR_INDEX);
    } else if (slot >= 0) {
      const long long page = P.num_slots <= 0xFFFFFFFFLL ? (long long)((unsigned)slot / (unsigned)P.page_size)
                                                         : slot / P.page_size;
      e = page * P.page_stride + (slot - page * P.page_size) * P.slot_stride;
    }
    dst[tid] = e;
  }
  __syncthreads();

  const Rows to = isq ? P.qo : P.ko;
  char *out = to_pages ? (isv ? P.vc : P.kc) + (KIND == TO_E4M3_PAGES ? 1 : 2) * ((long long)h * P.head_stride)
                       : to.p + 2 * ((long long)tok0 * to.ts + (long long)h * to.hs);
  f2 w0[H2], w1[H2];
  GV::unpack(w0, wa);
  GV::unpack(w1, wb);
  const f2 offset = pack2(P.offset, P.offset);
#pragma unroll
  for (int e = 0; e < H2; ++e) w0[e] = add2(w0[e], offset), w1[e] = add2(w1[e], offset);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f2 u[H2], v[H2];
    GV::unpack(u, a[i]);
    GV::unpack(v, b[i]);
    f2 ss = 0;
#pragma unroll
    for (int e = 0; e < H2; ++e) ss = fma2(u[e], u[e], fma2(v[e], v[e], ss));
    const float2 sp = unpack2(ss);
    float sum = sp.x + sp.y;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!active || tok0 + i >= P.T) continue;
    if (weight) {
      const float r = rsqrtf(fmaf(sum, 1.f / D, P.eps)) * inv;
      const f2 rr = pack2(r, r);
#pragma unroll
      for (int e = 0; e < H2; ++e) u[e] = mul2(u[e], mul2(rr, w0[e])), v[e] = mul2(v[e], mul2(rr, w1[e]));
    } else if (KIND == TO_E4M3_PAGES) {
      const f2 rr = pack2(inv, inv);
#pragma unroll
      for (int e = 0; e < H2; ++e) u[e] = mul2(u[e], rr), v[e] = mul2(v[e], rr);
    }
    if (rotates && !isv) {
      const float4 *t = cs + i * H2 * rlanes + lane;
#pragma unroll
      for (int e = 0; e < H2; ++e) {  // two pairs
        const float4 c4 = t[e * rlanes];
        const f2 c = pack2(c4.x, c4.y), s = pack2(c4.z, c4.w), ns = pack2(-c4.z, -c4.w);
        if (P.split) {
          const f2 x0 = u[e], x1 = v[e];
          u[e] = fma2(x0, c, mul2(x1, ns));
          v[e] = fma2(x0, s, mul2(x1, c));
        } else {  // elements 4e..4e+3 of the lane's 2V: (x0, x1), (x2, x3)
          f2 *y = e < H2 / 2 ? &u[2 * e] : &v[2 * e - H2];
          const float2 p = unpack2(y[0]), q = unpack2(y[1]);
          const f2 x0 = pack2(p.x, q.x), x1 = pack2(p.y, q.y);
          const float2 z0 = unpack2(fma2(x0, c, mul2(x1, ns))), z1 = unpack2(fma2(x0, s, mul2(x1, c)));
          y[0] = pack2(z0.x, z1.x);
          y[1] = pack2(z0.y, z1.y);
        }
      }
    }
    if (to_pages) {
      const long long e = dst[i];
      if (e < 0) continue;
      if (KIND == TO_E4M3_PAGES) {
        GV::store_e4m3(out + e + off0, u);
        GV::store_e4m3(out + e + off1, v);
      } else {
        GV::store_bf16(out + 2 * (e + off0), u);
        GV::store_bf16(out + 2 * (e + off1), v);
      }
    } else {
      char *row = out + 2 * (i * to.ts);
      GV::store_bf16(row + 2 * off0, u);
      GV::store_bf16(row + 2 * off1, v);
    }
  }
}

template <int D, int KIND, int V, int N>
static cudaError_t launch_n(Params &P, cudaStream_t s) {
  constexpr int LPR = D / (2 * V);
  // heads per block: the rows of about 256 threads, evenly over the blocks of a token
  const int most = 256 / LPR, blocks = (P.H + most - 1) / most;
  P.gh = (P.H + blocks - 1) / blocks;
  const int threads = (P.gh * LPR + 31) / 32 * 32;
  return launch_early(rope_kernel<D, KIND, V, N>, dim3((P.T + N - 1) / N, blocks), dim3(threads),
                      (size_t)N * (P.rot / 2) * sizeof(float2), s, P);
}

// More tokens a thread when the blocks fill the GPU several times over, else
// one (rows spread over more SMs).
template <int D, int KIND>
static cudaError_t launch_kind(Params &P, int sms, cudaStream_t s) {
  if (P.rot % 16 != 0) return launch_n<D, KIND, 4, 1>(P, s);
  const long long lanes = (long long)P.T * P.H * (D / 16);
  return lanes > 4LL * 2048 * sms ? launch_n<D, KIND, 8, 4>(P, s) : launch_n<D, KIND, 8, 1>(P, s);
}

template <int D>
static cudaError_t launch_d(Params &P, int kind, int sms, cudaStream_t s) {
  if (kind == TO_ROWS) return launch_kind<D, TO_ROWS>(P, sms, s);
  if (kind == TO_BF16_PAGES) return launch_kind<D, TO_BF16_PAGES>(P, sms, s);
  return launch_kind<D, TO_E4M3_PAGES>(P, sms, s);
}

static bool good_norm(const sv_head_norm *n) {
  return !n || (n->eps >= 0.f && n->eps < INFINITY && std::isfinite(n->weight_offset) &&
                paged::aligned(n->q_weight, 16) && paged::aligned(n->k_weight, 16));
}
static bool good_rotation(const sv_rotation *r, int T, int D) {
  if (!r || !r->phases) return true;
  return (r->positions || T == 0) && paged::aligned(r->phases, 8) && paged::aligned(r->positions, 4) &&
         r->rot_dim >= 8 && r->rot_dim % 8 == 0 && r->rot_dim <= D;
}

static void set_norm_rotation(Params &P, const sv_head_norm *n, const sv_rotation *r) {
  if (n) {
    P.qw = static_cast<const __nv_bfloat16 *>(n->q_weight);
    P.kw = static_cast<const __nv_bfloat16 *>(n->k_weight);
    P.eps = n->eps;
    P.offset = n->weight_offset;
  }
  if (r && r->phases) {
    P.phases = reinterpret_cast<const unsigned long long *>(r->phases);
    P.positions = r->positions;
    P.rot = r->rot_dim;
    P.split = r->interleaved ? 0 : 1;
  }
}

static Rows rows_of(const sv_rows *r) {
  return Rows{static_cast<char *>(r->ptr), (long long)r->token_stride, (long long)r->head_stride};
}

static sv_status run(Params &P, int D, int kind, int T, int Hq, int Hkv, int H, cudaStream_t s) {
  if (T == 0) return SV_OK;
  const int sms = device_sm_count();
  P.err = device_error_word();
  if (sms <= 0 || !P.err) return SV_ERR_CUDA;
  P.T = T;
  P.Hq = Hq;
  P.Hkv = Hkv;
  P.H = H;
  return from_cuda(D == 64 ? launch_d<64>(P, kind, sms, s)
                   : D == 128 ? launch_d<128>(P, kind, sms, s)
                              : launch_d<256>(P, kind, sms, s));
}

}  // namespace rope
}  // namespace sv

using namespace sv;

extern "C" {

sv_status rope_phases(const double *inv_freq, int n, uint64_t *phases_out) {
  if (n < 0 || (n > 0 && (!inv_freq || !phases_out))) return SV_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i])) return SV_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const double turns = inv_freq[i] / 6.283185307179586476925286766559;
    const double part = turns - std::floor(turns);  // [0, 1]
    const double hi = std::floor(std::ldexp(part, 32));
    const double lo = std::floor(std::ldexp(std::ldexp(part, 32) - hi, 32) + 0.5);
    phases_out[i] = ((uint64_t)hi << 32) + (uint64_t)lo;
  }
  return SV_OK;
}

sv_status qk_norm_rope(const sv_rows *q, const sv_rows *k, const sv_rows *q_out, const sv_rows *k_out,
                       const sv_head_norm *norm, const sv_rotation *rot, int T, int Hq, int Hkv, int D,
                       sv_stream_t stream) {
  if (T < 0 || Hq < 1 || Hkv < 1 || D < 1) return SV_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return SV_ERR_UNSUPPORTED;
  if (Hq > 4096 || Hkv > 4096 || (long long)T * (Hq + Hkv) > 0x7fffffffLL) return SV_ERR_UNSUPPORTED;
  for (const sv_rows *r : {q, k, q_out, k_out})
    if (!paged::good_rows(r, T)) return SV_ERR_INVALID_ARG;
  if (!rope::good_norm(norm) || !rope::good_rotation(rot, T, D)) return SV_ERR_INVALID_ARG;
  rope::Params P{};
  P.q = rope::rows_of(q);
  P.k = rope::rows_of(k);
  P.qo = rope::rows_of(q_out);
  P.ko = rope::rows_of(k_out);
  rope::set_norm_rotation(P, norm, rot);
  return rope::run(P, D, rope::TO_ROWS, T, Hq, Hkv, Hq + Hkv, reinterpret_cast<cudaStream_t>(stream));
}

sv_status paged_kv_append(const sv_rows *q, const sv_rows *q_out, const sv_rows *k, const sv_rows *v,
                          const sv_paged_kv *cache, const int64_t *slots, const sv_head_norm *norm,
                          const sv_rotation *rot, int T, int Hq, int Hkv, int D, sv_stream_t stream) {
  if (T < 0 || Hkv < 1 || D < 1 || (q && Hq < 1)) return SV_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return SV_ERR_UNSUPPORTED;
  const int heads = q ? Hq : 0;
  if (heads > 4096 || Hkv > 4096 || (long long)T * ((long long)heads + 2 * Hkv) > 0x7fffffffLL)
    return SV_ERR_UNSUPPORTED;
  if (!paged::good_rows(k, T) || !paged::good_rows(v, T)) return SV_ERR_INVALID_ARG;
  if (q && (!paged::good_rows(q, T) || !paged::good_rows(q_out, T))) return SV_ERR_INVALID_ARG;
  const sv_status cs = paged::check_cache(cache, D);
  if (cs != SV_OK) return cs;
  if ((!slots && T > 0) || !paged::aligned(slots, 8)) return SV_ERR_INVALID_ARG;
  if (!rope::good_norm(norm) || !rope::good_rotation(rot, T, D)) return SV_ERR_INVALID_ARG;
  rope::Params P{};
  if (q) {
    P.q = rope::rows_of(q);
    P.qo = rope::rows_of(q_out);
  }
  P.k = rope::rows_of(k);
  P.v = rope::rows_of(v);
  rope::set_norm_rotation(P, norm, rot);
  P.slots = reinterpret_cast<const long long *>(slots);
  P.kc = static_cast<char *>(cache->k);
  P.vc = static_cast<char *>(cache->v);
  P.ks = cache->k_scale;
  P.vs = cache->v_scale;
  P.page_stride = cache->page_stride;
  P.slot_stride = cache->slot_stride;
  P.head_stride = cache->head_stride;
  P.page_size = cache->page_size;
  P.num_slots = cache->num_pages * cache->page_size;
  return rope::run(P, D, cache->dtype == SV_E4M3 ? rope::TO_E4M3_PAGES : rope::TO_BF16_PAGES, T, heads,
                   Hkv, heads + 2 * Hkv, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
