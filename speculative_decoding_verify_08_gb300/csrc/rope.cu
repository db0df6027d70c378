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
//    kind, weights and strides are worked out once, a row costs one address
//    step, and the N rows' loads are all in flight before anything is computed.
//    A block holds neighbouring heads, so its loads of a token are one run of
//    memory.
//  * D/(2V) lanes share a row.  A lane of a half-split rotation holds V elements of
//    the first half and their V partners of the second, so that a pair never
//    leaves its lane; V = 8 (16-byte accesses) unless rot_dim is no multiple
//    of 16 (V = 4).
//  * The sines of a block's tokens are made once, in shared memory, while the
//    rows' loads are in flight, and serve all its heads.
//  * The angle is an integer: position times a 64-bit fraction of a turn wraps
//    at whole turns by itself, so a far position loses nothing and no 64-bit
//    floating-point arithmetic is needed.
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

__device__ __forceinline__ uint32_t e4m3x4(const float *y) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Cosine and sine of position * phase / 2^64 turns.  The product's upper 32
// bits, as a signed fraction of a turn, are off by 2^-33 turns at most, below
// the fp32 rounding of the fraction itself.
__device__ __forceinline__ float2 turn(int pos, unsigned long long phase) {
  const unsigned long long f = (unsigned long long)(long long)pos * phase;
  float s, c;
  sincospif((float)(int)(f >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ void unpack(float *y, uint4 v) {
  y[0] = bf16lo(v.x), y[1] = bf16hi(v.x), y[2] = bf16lo(v.y), y[3] = bf16hi(v.y);
  y[4] = bf16lo(v.z), y[5] = bf16hi(v.z), y[6] = bf16lo(v.w), y[7] = bf16hi(v.w);
}
__device__ __forceinline__ void unpack(float *y, uint2 v) {
  y[0] = bf16lo(v.x), y[1] = bf16hi(v.x), y[2] = bf16lo(v.y), y[3] = bf16hi(v.y);
}
__device__ __forceinline__ void store_bf16(char *p, const float (&y)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                             pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}
__device__ __forceinline__ void store_bf16(char *p, const float (&y)[4]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}
__device__ __forceinline__ void store_e4m3(char *p, const float (&y)[8]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(e4m3x4(y), e4m3x4(y + 4));
}
__device__ __forceinline__ void store_e4m3(char *p, const float (&y)[4]) {
  *reinterpret_cast<uint32_t *>(p) = e4m3x4(y);
}

template <int V>
struct Group;
template <>
struct Group<8> {
  using type = uint4;
};
template <>
struct Group<4> {
  using type = uint2;
};

template <int D, int KIND, int V, int N>
__global__ void __launch_bounds__(MAX_THREADS) rope_kernel(const Params P) {
  using G = typename Group<V>::type;
  constexpr int LPR = D / (2 * V);  // lanes per row
  extern __shared__ __align__(16) float2 cs[];  // [N][rot/2] cosine and sine
  __shared__ long long dst[N];                  // element of the token's slot, or -1
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid % LPR, grp = tid / LPR;
  const int head = blockIdx.y * P.gh + grp;
  const bool active = grp < P.gh && head < P.H;
  const int tok0 = blockIdx.x * N;
  const bool isq = head < P.Hq, isv = head >= P.Hq + P.Hkv;
  const int h = isq ? head : isv ? head - P.Hq - P.Hkv : head - P.Hq;
  const bool rotates = lane < P.rot / (2 * V);
  // first elements of this lane's two groups of V
  const int off0 = (P.split && rotates) ? V * lane : 2 * V * lane;
  const int off1 = (P.split && rotates) ? P.rot / 2 + V * lane : 2 * V * lane + V;

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
  float w0[V], w1[V];
  if (active && weight) {
    unpack(w0, *reinterpret_cast<const G *>(weight + off0));
    unpack(w1, *reinterpret_cast<const G *>(weight + off1));
#pragma unroll
    for (int i = 0; i < V; ++i) w0[i] += P.offset, w1[i] += P.offset;
  }

  const int half = P.rot / 2;
#pragma unroll
  for (int t = 0; t < N; ++t) {
    if (tok0 + t >= P.T) break;
    const int pos = half ? P.positions[tok0 + t] : 0;
    for (int i = tid; i < half; i += blockDim.x) cs[t * half + i] = turn(pos, P.phases[i]);
  }
  if (KIND != TO_ROWS && tid < N && tok0 + tid < P.T) {
    const long long s = P.slots[tok0 + tid];
    long long e = -1;
    if (s >= P.num_slots) {
      atomicOr(P.err, ERR_INDEX);
    } else if (s >= 0) {
      const long long page = P.num_slots <= 0xFFFFFFFFLL ? (long long)((unsigned)s / (unsigned)P.page_size)
                                                         : s / P.page_size;
      e = page * P.page_stride + (s - page * P.page_size) * P.slot_stride;
    }
    dst[tid] = e;
  }
  __syncthreads();

  const bool to_pages = KIND != TO_ROWS && !isq;
  const Rows to = isq ? P.qo : P.ko;
  char *out = to_pages ? (isv ? P.vc : P.kc) + (KIND == TO_E4M3_PAGES ? 1 : 2) * ((long long)h * P.head_stride)
                       : to.p + 2 * ((long long)tok0 * to.ts + (long long)h * to.hs);
  float inv = 1.f;
  if (KIND == TO_E4M3_PAGES && active && to_pages) {
    const float *sp = isv ? P.vs : P.ks;
    if (sp) inv = 1.f / sp[h];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float u[V], v[V];
    unpack(u, a[i]);
    unpack(v, b[i]);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) ss = fmaf(u[e], u[e], fmaf(v[e], v[e], ss));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!active || tok0 + i >= P.T) continue;
    if (weight) {
      const float r = rsqrtf(fmaf(ss, 1.f / D, P.eps));
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] *= r * w0[e], v[e] *= r * w1[e];
    }
    if (rotates && !isv) {
      const float4 *t = reinterpret_cast<const float4 *>(cs + i * half + V * lane);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {  // (cos, sin) of two pairs
        const float4 c = t[e];
        if (P.split) {
          const float u0 = u[2 * e], u1 = u[2 * e + 1], v0 = v[2 * e], v1 = v[2 * e + 1];
          u[2 * e] = u0 * c.x - v0 * c.y;
          v[2 * e] = u0 * c.y + v0 * c.x;
          u[2 * e + 1] = u1 * c.z - v1 * c.w;
          v[2 * e + 1] = u1 * c.w + v1 * c.z;
        } else {
          float *y = e < V / 4 ? u : v;
          const int k = e < V / 4 ? 4 * e : 4 * e - V;
          const float y0 = y[k], y1 = y[k + 1], y2 = y[k + 2], y3 = y[k + 3];
          y[k] = y0 * c.x - y1 * c.y;
          y[k + 1] = y0 * c.y + y1 * c.x;
          y[k + 2] = y2 * c.z - y3 * c.w;
          y[k + 3] = y2 * c.w + y3 * c.z;
        }
      }
    }
    if (to_pages) {
      const long long e = dst[i];
      if (e < 0) continue;
      if (KIND == TO_E4M3_PAGES) {
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] *= inv, v[j] *= inv;
        store_e4m3(out + e + off0, u);
        store_e4m3(out + e + off1, v);
      } else {
        store_bf16(out + 2 * (e + off0), u);
        store_bf16(out + 2 * (e + off1), v);
      }
    } else {
      store_bf16(out + 2 * (i * to.ts + off0), u);
      store_bf16(out + 2 * (i * to.ts + off1), v);
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

// Four tokens a thread when the blocks fill the GPU several times over (four
// rows' loads in flight), else one (rows spread over more SMs).
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
static bool good_rotation(const sv_rotation *r, int D) {
  if (!r || !r->phases) return true;
  return r->positions && paged::aligned(r->phases, 8) && paged::aligned(r->positions, 4) &&
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
  if (!rope::good_norm(norm) || !rope::good_rotation(rot, D)) return SV_ERR_INVALID_ARG;
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
  if (!rope::good_norm(norm) || !rope::good_rotation(rot, D)) return SV_ERR_INVALID_ARG;
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
