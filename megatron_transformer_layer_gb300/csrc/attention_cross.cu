// Entry points of the attention to keys of another length: argument checks and
// the launch order.  The kernels are in attention_cross_fwd.cu and
// attention_cross_bwd.cu.
#include <cuda_runtime.h>

#include "mc_layer_internal.h"

namespace mc {

int launch_attention_cross_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               uint16_t* o, float* lse, const mc_cross_attention& c, int* status,
                               cudaStream_t st);
size_t attention_cross_ws_bytes(const mc_cross_attention& c);
int launch_attention_cross_bwd(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               const uint16_t* o, const float* lse, const uint16_t* dout,
                               uint16_t* dq, uint16_t* dk, uint16_t* dv, float* delta,
                               const mc_cross_attention& c, uint8_t* ws, size_t ws_bytes,
                               int* status, cudaStream_t st);

namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check_cross(const mc_cross_attention* c) {
  if (!c) return MC_ERR_NULLPTR;
  if (c->sequences < 1 || c->heads < 1 || c->kv_heads < 1 || c->q_rows < 1 || c->kv_rows < 1 ||
      c->max_q < 0 || c->max_kv < 0 || c->heads % c->kv_heads)
    return MC_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return MC_ERR_UNSUPPORTED;
  // a group's heads of one query fill a tile at most
  if (c->heads / c->kv_heads > 128) return MC_ERR_UNSUPPORTED;
  const int64_t a = static_cast<int64_t>(c->heads) * c->head_dim,
                akv = static_cast<int64_t>(c->kv_heads) * c->head_dim;
  if (a > (1 << 20) || c->sequences > (1 << 20) || c->q_rows > (1 << 28) || c->kv_rows > (1 << 28))
    return MC_ERR_UNSUPPORTED;
  if (c->ld_q < a || c->ld_o < a || c->ld_kv < akv) return MC_ERR_SHAPE;
  if (c->ld_q % 8 || c->ld_o % 8 || c->ld_kv % 8) return MC_ERR_ALIGN;
  // (a group's heads are a dimension of the tensor maps, whose strides are
  // multiples of one another)
  if (c->heads != c->kv_heads && (c->ld_q % c->head_dim || c->ld_o % c->head_dim))
    return MC_ERR_ALIGN;
  // (strides of the tensor maps stay below 2^40 bytes)
  if (c->ld_q > (1ll << 38) / c->q_rows || c->ld_o > (1ll << 38) / c->q_rows ||
      c->ld_kv > (1ll << 38) / c->kv_rows)
    return MC_ERR_UNSUPPORTED;
  if ((!c->q_offsets && c->q_rows % c->sequences) || (!c->kv_offsets && c->kv_rows % c->sequences))
    return MC_ERR_SHAPE;
  if (!aligned(c->q_offsets, 4) || !aligned(c->q_lens, 4) || !aligned(c->kv_offsets, 4) ||
      !aligned(c->kv_lens, 4))
    return MC_ERR_ALIGN;
  if (!(c->scale == 0.f || (c->scale >= 0x1p-16f && c->scale <= 0x1p16f))) return MC_ERR_ARGUMENT;
  // items, and twice of them (the launches' shares), are counted in 32 bits
  const int64_t pq = 128 / (c->heads / c->kv_heads);
  auto most = [&](const int32_t* off, int64_t rows, int64_t bound) {
    return !off ? rows / c->sequences : bound > 0 && bound < rows ? bound : rows;
  };
  const int64_t nqb = (most(c->q_offsets, c->q_rows, c->max_q) + pq - 1) / pq,
                nkb = (most(c->kv_offsets, c->kv_rows, c->max_kv) + 127) / 128;
  const int64_t longest = nqb > nkb ? nqb : nkb;
  if (longest * c->sequences * c->kv_heads >= (1ll << 30)) return MC_ERR_UNSUPPORTED;
  return MC_OK;
}

}  // namespace
}  // namespace mc

using namespace mc;

extern "C" {

int mc_attention_forward_cross(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               uint16_t* o, float* lse, const mc_cross_attention* cross,
                               int* status, void* stream) {
  const int rc = check_cross(cross);
  if (rc != MC_OK) return rc;
  if (!q || !k || !v || !o || !lse) return MC_ERR_NULLPTR;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return MC_ERR_ALIGN;
  return launch_attention_cross_fwd(q, k, v, o, lse, *cross, status,
                                    static_cast<cudaStream_t>(stream));
}

size_t mc_attention_backward_cross_ws_bytes(const mc_cross_attention* cross) {
  return check_cross(cross) == MC_OK ? attention_cross_ws_bytes(*cross) : 0;
}

int mc_attention_backward_cross(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                const uint16_t* o, const float* lse, const uint16_t* dout,
                                uint16_t* dq, uint16_t* dk, uint16_t* dv, float* delta,
                                const mc_cross_attention* cross, void* ws, size_t ws_bytes,
                                int* status, void* stream) {
  const int rc = check_cross(cross);
  if (rc != MC_OK) return rc;
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !delta || !ws)
    return MC_ERR_NULLPTR;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
      !aligned(lse, 4) || !aligned(delta, 4) || !aligned(ws, 16))
    return MC_ERR_ALIGN;
  const size_t need = attention_cross_ws_bytes(*cross);
  if (need == 0) return MC_ERR_UNSUPPORTED;
  if (ws_bytes < need) return MC_ERR_WORKSPACE;
  return launch_attention_cross_bwd(q, k, v, o, lse, dout, dq, dk, dv, delta, *cross,
                                    static_cast<uint8_t*>(ws), ws_bytes, status,
                                    static_cast<cudaStream_t>(stream));
}

}  // extern "C"
