// Test harness: the product's tensor-core kernels, launched as the library does, but with a limit of the caller's on every
// wait and, where `starve` is set, with copies of the codes that are half as high as the barriers expect.  Those copies
// land, in bounds, and the barriers of the operands never complete: every wait that depends on them has to run out.
#include "../int4_expert_ffn_top_b200/csrc/linear_api.cu"

extern "C" int linear8_waits(int kind, const moe_linear8* W, const int8_t* q, int64_t ldq, const float* qscale, int32_t T,
                             void* out, int32_t* err_word, int64_t timeout_ns, int starve, void* stream) {
  l8::LinArgs lin{W->codes, W->ld, W->scale, W->bias, q, ldq, qscale, T, W->out_dim, 0, out, 0};
  int dev = 0;
  const int nsm = multiprocessors(&dev), rows = kind ? l8::kGM : 2 * l8::kGM, bn = kind ? 32 : 64;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  l8::GemmMaps maps;
  l8::GemmArgs a{};
  if (nsm < 1 || !make_args(&maps, &a, lin, W->in_dim, rows, bn, 32, err_word)) return MOE_ERR_CUDA;
  a.timeout_ns = timeout_ns;
  if (starve && !codes_map(&maps.q, q, W->in_dim, T, ldq, 16)) return MOE_ERR_CUDA;
  return kind ? launch_split_mode<32, 0>(maps, a, starve > 1 ? 1 : 2, dev, st) : launch_gemm_mode<64, 0>(maps, a, nsm, dev, st);
}
