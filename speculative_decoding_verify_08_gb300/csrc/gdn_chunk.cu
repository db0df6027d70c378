// gdn_chunk.cu -- the gated delta rule over packed chunks of new tokens, from
// the states of a pool and back into it.
#include "gdn_pool.cuh"

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
  return gdn::launch_tokens(P, dk, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
