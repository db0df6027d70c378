// rope.cu -- per-head RMS norm and position rotation of query and key rows,
// and their (and the values') way into a paged cache, in one pass.
//
// Row x of D elements of one (token, head):
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset)
//   (u, v) <- (u cos a - v sin a, u sin a + v cos a),  a = position * inv_freq[pair]
// computed in fp32 and rounded once.
//
// What bounds it: every row is read once and written once (about 60 fp32
// instructions per 16 bytes read), so HBM at many tokens and the launch at
// few.  Hence:
//  * Rows are taken in (token, head) order, D/8 lanes a row, so a block's
//    rows are a run of memory and consecutive blocks stream it; each thread
//    has the loads of its U rows in flight before it computes.
//  * A lane of a half-split rotation holds four elements of the first half and
//    their four partners of the second, so a pair never leaves its lane.
//  * The sines of a block's few tokens are made once, in shared memory, while
//    the rows' loads are in flight, and serve all heads.
//  * The angle is an integer: position times a 64-bit fraction of a turn wraps
//    at whole turns by itself, so a far position loses nothing and no 64-bit
//    floating-point arithmetic is needed.
#include <cuda_fp8.h>

#include <cmath>

#include "paged.cuh"

namespace sv {
namespace rope {

constexpr int THREADS = 256;

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
  unsigned magic;     // ceil(2^32 / H)
  int span;           // tokens that a block's rows can touch
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

// U rows per thread: 4 when the rows fill the GPU several times over (four
// 16-byte loads in flight a thread), else 1 (the rows spread over more SMs).
template <int D, int KIND, int U>
__global__ void __launch_bounds__(THREADS) rope_kernel(const Params P) {
  constexpr int LPR = D / 8;           // lanes per row
  constexpr int RPP = THREADS / LPR;   // rows per pass
  extern __shared__ __align__(16) uint8_t smem[];
  float *wt = reinterpret_cast<float *>(smem);                         // [2][D] weights
  long long *dst = reinterpret_cast<long long *>(smem + 2 * D * 4);    // [span] element, or -1
  float2 *cs = reinterpret_cast<float2 *>(dst + (P.span + 1) / 2 * 2);  // [span][rot/2]
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid % LPR;
  const unsigned total = (unsigned)P.T * (unsigned)P.H;
  const unsigned r0 = blockIdx.x * (unsigned)(RPP * U);
  const int tok0 = (int)(r0 / (unsigned)P.H);
  const int h0 = (int)(r0 - (unsigned)tok0 * (unsigned)P.H);
  const bool rotates = lane < P.rot / 8;
  // first elements of this lane's two groups of four
  const int off0 = (P.split && rotates) ? 4 * lane : 8 * lane;
  const int off1 = (P.split && rotates) ? P.rot / 2 + 4 * lane : 8 * lane + 4;

  uint2 a[U], b[U];
  int tl[U], hd[U];
  bool have[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int local = tid / LPR + u * RPP;
    have[u] = r0 + (unsigned)local < total;
    tl[u] = (int)__umulhi((unsigned)(h0 + local), P.magic);
    hd[u] = h0 + local - tl[u] * P.H;
    a[u] = b[u] = make_uint2(0u, 0u);
    if (have[u]) {
      const Rows &src = hd[u] < P.Hq ? P.q : hd[u] < P.Hq + P.Hkv ? P.k : P.v;
      const int h = hd[u] < P.Hq ? hd[u] : hd[u] < P.Hq + P.Hkv ? hd[u] - P.Hq : hd[u] - P.Hq - P.Hkv;
      const char *x = src.p + 2 * ((long long)(tok0 + tl[u]) * src.ts + (long long)h * src.hs);
      if (P.split) {
        a[u] = *reinterpret_cast<const uint2 *>(x + 2 * off0);
        b[u] = *reinterpret_cast<const uint2 *>(x + 2 * off1);
      } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(x + 16 * lane);
        a[u] = make_uint2(v.x, v.y);
        b[u] = make_uint2(v.z, v.w);
      }
    }
  }

  const int ntok = imin(P.span, P.T - tok0);
  const int half = P.rot / 2;
  for (int i = tid; i < ntok * half; i += THREADS) {
    const int t = i / half;
    cs[i] = turn(P.positions[tok0 + t], P.phases[i - t * half]);
  }
  for (int i = tid; i < 2 * D; i += THREADS) {
    const __nv_bfloat16 *w = i < D ? P.qw : P.kw;
    wt[i] = w ? __bfloat162float(w[i % D]) + P.offset : 1.f;
  }
  if (KIND != TO_ROWS) {
    for (int i = tid; i < ntok; i += THREADS) {
      const long long s = P.slots[tok0 + i];
      long long e = -1;
      if (s >= P.num_slots) {
        atomicOr(P.err, ERR_INDEX);
      } else if (s >= 0) {
        const long long page = P.num_slots <= 0xFFFFFFFFLL ? (long long)((unsigned)s / (unsigned)P.page_size)
                                                           : s / P.page_size;
        e = page * P.page_stride + (s - page * P.page_size) * P.slot_stride;
      }
      dst[i] = e;
    }
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool isq = hd[u] < P.Hq, isv = hd[u] >= P.Hq + P.Hkv;
    float y[8] = {bf16lo(a[u].x), bf16hi(a[u].x), bf16lo(a[u].y), bf16hi(a[u].y),
                  bf16lo(b[u].x), bf16hi(b[u].x), bf16lo(b[u].y), bf16hi(b[u].y)};
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!have[u]) continue;
    if (!isv) {
      if (isq ? P.qw != nullptr : P.kw != nullptr) {
        const float r = rsqrtf(fmaf(ss, 1.f / D, P.eps));
        const float *w = wt + (isq ? 0 : D);
        const float4 w0 = *reinterpret_cast<const float4 *>(w + off0);
        const float4 w1 = *reinterpret_cast<const float4 *>(w + off1);
        y[0] *= r * w0.x, y[1] *= r * w0.y, y[2] *= r * w0.z, y[3] *= r * w0.w;
        y[4] *= r * w1.x, y[5] *= r * w1.y, y[6] *= r * w1.z, y[7] *= r * w1.w;
      }
      if (rotates) {
        const float4 *t = reinterpret_cast<const float4 *>(cs + tl[u] * half + 4 * lane);
        const float4 c01 = t[0], c23 = t[1];  // (cos, sin) of four pairs
        const float c[4] = {c01.x, c01.z, c23.x, c23.z}, s[4] = {c01.y, c01.w, c23.y, c23.w};
        float z[8];
        if (P.split) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = y[i] * c[i] - y[4 + i] * s[i];
            z[4 + i] = y[i] * s[i] + y[4 + i] * c[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[2 * i] = y[2 * i] * c[i] - y[2 * i + 1] * s[i];
            z[2 * i + 1] = y[2 * i] * s[i] + y[2 * i + 1] * c[i];
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = z[i];
      }
    }
    char *out;
    if (isq || KIND == TO_ROWS) {
      const Rows &d = isq ? P.qo : P.ko;
      out = d.p + 2 * ((long long)(tok0 + tl[u]) * d.ts + (long long)(isq ? hd[u] : hd[u] - P.Hq) * d.hs);
    } else {
      const long long e = dst[tl[u]];
      if (e < 0) continue;
      const int h = isv ? hd[u] - P.Hq - P.Hkv : hd[u] - P.Hq;
      out = (isv ? P.vc : P.kc) + (KIND == TO_E4M3_PAGES ? 1 : 2) * (e + (long long)h * P.head_stride);
      if (KIND == TO_E4M3_PAGES) {
        const float *sp = isv ? P.vs : P.ks;
        const float inv = sp ? 1.f / sp[h] : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= inv;
        *reinterpret_cast<uint32_t *>(out + off0) = e4m3x4(y);
        *reinterpret_cast<uint32_t *>(out + off1) = e4m3x4(y + 4);
        continue;
      }
    }
    const uint2 z0 = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    const uint2 z1 = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    if (P.split) {
      *reinterpret_cast<uint2 *>(out + 2 * off0) = z0;
      *reinterpret_cast<uint2 *>(out + 2 * off1) = z1;
    } else {
      *reinterpret_cast<uint4 *>(out + 16 * lane) = make_uint4(z0.x, z0.y, z1.x, z1.y);
    }
  }
}

template <int D, int KIND, int U>
static cudaError_t launch_u(Params &P, cudaStream_t s) {
  constexpr int RB = THREADS / (D / 8) * U;
  P.span = imin((RB - 1) / P.H + 2, P.T);
  const unsigned total = (unsigned)P.T * (unsigned)P.H;
  const size_t smem = 2 * D * 4 + (size_t)(P.span + 1) / 2 * 16 + (size_t)P.span * (P.rot / 2) * 8;
  return launch(rope_kernel<D, KIND, U>, dim3((total + RB - 1) / RB), dim3(THREADS), smem, s, P);
}

template <int D, int KIND>
static cudaError_t launch_kind(Params &P, int sms, cudaStream_t s) {
  const long long rows = (long long)P.T * P.H;
  const long long pass = THREADS / (D / 8);
  return rows > 8 * pass * sms ? launch_u<D, KIND, 4>(P, s) : launch_u<D, KIND, 1>(P, s);
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
  P.magic = (unsigned)((0x100000000ULL + (unsigned)H - 1) / (unsigned)H);
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
