// Entry points of the attention over interval masks: argument checks and the
// launch order.  The kernels are in attention_opt_fwd.cu and
// attention_opt_bwd.cu; the delta = rowsum(dO O) pre-pass is attention.cu's.
// It takes the stored bf16 O, each element of which is off by up to 2^-8 of
// itself, and sums in 32 bits: the exact sum of P dP would need every score of a
// row before its first dz, a pass of its own over S and dP.  The error it leaves
// in dz shows most in rows that see few keys, where O averages little.
#include <cuda_runtime.h>

#include "mc_layer_internal.h"

namespace mc {

int launch_attention_opt_fwd(const uint16_t* qkv, uint16_t* o, float* lse, int b, int s, int H,
                             int d, const mc_attention_options& opt, int* status,
                             cudaStream_t st);
int launch_attention_opt_bwd(const uint16_t* qkv, const float* lse, const uint16_t* dout,
                             uint16_t* dqkv, const float* delta, int b, int s, int H, int d,
                             const mc_attention_options& opt, uint8_t* ds_tiles, int* status,
                             cudaStream_t st);

namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check_shape(int b, int s, int H, int d) {
  if (b < 1 || s < 1 || H < 1) return MC_ERR_SHAPE;
  if (d != 64 && d != 128) return MC_ERR_UNSUPPORTED;
  // the limits of the mask's tables, and 3 * heads * head_dim <= 2^20 as in the layer
  if (H > 65535 || b > 65535 || static_cast<int64_t>(b) * s > (1 << 24) ||
      3ll * H * d > (1 << 20))
    return MC_ERR_UNSUPPORTED;
  return MC_OK;
}

}  // namespace

int check_attention_options(const mc_attention_options* opt) {
  if (!opt || !opt->key_lo || !opt->key_hi || !opt->tables) return MC_ERR_NULLPTR;
  if (!aligned(opt->key_lo, 4) || !aligned(opt->key_hi, 4) || !aligned(opt->tables, 16) ||
      !aligned(opt->slopes, 4))
    return MC_ERR_ALIGN;
  // (the range in which the cap's forms hold in 32 bits)
  if (!(opt->softcap == 0.f || (opt->softcap >= 0x1p-16f && opt->softcap <= 0x1p16f)))
    return MC_ERR_ARGUMENT;
  return MC_OK;
}

int launch_attention_forward_opt(const uint16_t* qkv, uint16_t* o, float* lse, int b, int s, int H,
                                 int d, const mc_attention_options& opt, int* status,
                                 cudaStream_t st) {
  const int rc = check_shape(b, s, H, d);
  if (rc != MC_OK) return rc;
  if (!qkv || !o || !lse) return MC_ERR_NULLPTR;
  if (!aligned(qkv, 16) || !aligned(o, 16) || !aligned(lse, 4)) return MC_ERR_ALIGN;
  return launch_attention_opt_fwd(qkv, o, lse, b, s, H, d, opt, status, st);
}

int launch_attention_backward_opt(const uint16_t* qkv, const uint16_t* o, const float* lse,
                                  const uint16_t* dout, uint16_t* dqkv, float* delta, int b, int s,
                                  int H, int d, const mc_attention_options& opt, uint8_t* ds_tiles,
                                  int* status, cudaStream_t st) {
  int rc = check_shape(b, s, H, d);
  if (rc != MC_OK) return rc;
  if (!qkv || !o || !lse || !dout || !dqkv || !delta) return MC_ERR_NULLPTR;
  if (!aligned(qkv, 16) || !aligned(o, 16) || !aligned(dout, 16) || !aligned(dqkv, 16) ||
      !aligned(lse, 4) || !aligned(delta, 4) || !aligned(ds_tiles, 16))
    return MC_ERR_ALIGN;
  rc = launch_attention_delta(o, dout, delta, b, s, H, d, st);
  if (rc != MC_OK) return rc;
  return launch_attention_opt_bwd(qkv, lse, dout, dqkv, delta, b, s, H, d, opt, ds_tiles, status,
                                  st);
}

}  // namespace mc

using namespace mc;

extern "C" {

int mc_attention_forward_opt(const uint16_t* qkv, uint16_t* o, float* lse, int32_t micro_batch,
                             int32_t seq_len, int32_t heads, int32_t head_dim,
                             const mc_attention_options* options, int* status, void* stream) {
  const int rc = check_attention_options(options);
  if (rc != MC_OK) return rc;
  return launch_attention_forward_opt(qkv, o, lse, micro_batch, seq_len, heads, head_dim, *options,
                                      status, static_cast<cudaStream_t>(stream));
}

size_t mc_attention_backward_opt_ws_bytes(int32_t micro_batch, int32_t seq_len, int32_t heads,
                                          int32_t head_dim, const mc_attention_options* options) {
  if (!options || check_shape(micro_batch, seq_len, heads, head_dim) != MC_OK) return 0;
  return static_cast<size_t>(
      attention_opt_ds_bytes(micro_batch, seq_len, heads, options->causal != 0));
}

int mc_attention_backward_opt(const uint16_t* qkv, const uint16_t* o, const float* lse,
                              const uint16_t* dout, uint16_t* dqkv, float* delta,
                              int32_t micro_batch, int32_t seq_len, int32_t heads,
                              int32_t head_dim, const mc_attention_options* options,
                              void* ds_workspace, size_t ds_workspace_bytes, int* status,
                              void* stream) {
  int rc = check_attention_options(options);
  if (rc != MC_OK) return rc;
  rc = check_shape(micro_batch, seq_len, heads, head_dim);
  if (rc != MC_OK) return rc;
  if (ds_workspace && ds_workspace_bytes < mc_attention_backward_opt_ws_bytes(
                                               micro_batch, seq_len, heads, head_dim, options))
    return MC_ERR_WORKSPACE;
  return launch_attention_backward_opt(qkv, o, lse, dout, dqkv, delta, micro_batch, seq_len, heads,
                                       head_dim, *options, static_cast<uint8_t*>(ds_workspace),
                                       status, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
