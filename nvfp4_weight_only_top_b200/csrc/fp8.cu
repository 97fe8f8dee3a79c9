// C ABI of the block-scaled E4M3 operators: host-side validation and the launches (fp8_quant.cu,
// fp8_matmul.cu).
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "internal.h"
#include "moe_nvfp4.h"

namespace {

constexpr int kMaxWidth = 65536;

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int bad(const char* what, long long v) {
  char msg[160];
  snprintf(msg, sizeof(msg), "%s (got %lld)", what, v);
  return moe::api_fail(MOE_NVFP4_ERR_INVALID_ARG, msg);
}

int done(int rc, const char* what) {
  if (rc < 0) return moe::api_cuda_fail(-rc, what);
  moe::api_set_launches(rc);
  return MOE_NVFP4_OK;
}

// Inputs of a row: a multiple of 16 (16-byte rows of E4M3, 32-byte rows of BF16).
int check_width(int32_t K, const char* what) {
  if (K >= 16 && K % 16 == 0 && K <= kMaxWidth) return MOE_NVFP4_OK;
  char msg[160];
  snprintf(msg, sizeof(msg), "%s = %d must be a multiple of 16 in 16..%d", what, K, kMaxWidth);
  return moe::api_fail(MOE_NVFP4_ERR_UNSUPPORTED, msg);
}

// Rows, and the device.
int check_rows(int64_t rows, const char* what) {
  moe::api_set_launches(0);
  if (rows < 0) return bad(what, rows);
  if (rows >= (int64_t)1 << 26) return moe::api_fail(MOE_NVFP4_ERR_UNSUPPORTED, "too many rows (limit 2^26)");
  return MOE_NVFP4_OK;
}

int check_pointers(const void* in, const void* q, const void* scales) {
  if (!in || !q || !scales) return moe::api_fail(MOE_NVFP4_ERR_INVALID_ARG, "a pointer argument is NULL");
  if (!al(in, 16) || !al(q, 16) || !al(scales, 4))
    return moe::api_fail(MOE_NVFP4_ERR_INVALID_ARG, "values and codes must be 16-byte aligned, scales 4-byte aligned");
  return MOE_NVFP4_OK;
}

// MOE_NVFP4_FP8_TILE, for comparisons: 64, 128 or 256, or 64xP or 128xP with P = 1..8 CTAs a tile.
int check_tile(moe::Fp8Tile* tile) {
  const char* s = getenv("MOE_NVFP4_FP8_TILE");
  if (!s || !*s) return MOE_NVFP4_OK;
  for (const int bn : {64, 128, 256}) {
    char text[8];
    const int n = snprintf(text, sizeof(text), "%d", bn);
    if (strncmp(s, text, n) != 0) continue;
    if (s[n] == 0) {
      tile->bn = bn;
      return MOE_NVFP4_OK;
    }
    if (bn < 256 && s[n] == 'x' && s[n + 1] >= '1' && s[n + 1] <= '0' + moe::kFp8MaxParts && s[n + 2] == 0) {
      tile->bn = bn;
      tile->parts = s[n + 1] - '0';
      return MOE_NVFP4_OK;
    }
  }
  char msg[160];
  snprintf(msg, sizeof(msg), "MOE_NVFP4_FP8_TILE=%.40s is not 64, 128, 256, 64xP or 128xP with P in 1..%d", s,
           moe::kFp8MaxParts);
  return moe::api_fail(MOE_NVFP4_ERR_INVALID_ARG, msg);
}

}  // namespace

extern "C" {

int moe_nvfp4_fp8_quantize(const void* x_dev, int64_t T, int32_t K, const int32_t* inv_dev, int32_t k, void* q_dev,
                           float* scales_dev, void* stream) {
  int rc = check_rows(T, "T is negative");
  if (rc || (rc = check_width(K, "K"))) return rc;
  if (k < 1 || k > 32) return bad("k outside 1..32", k);
  if (T > 0 && !inv_dev && k != 1) return bad("k must be 1 without inv", k);   // (an empty inv has no address)
  if (T * k >= (int64_t)1 << 26) return moe::api_fail(MOE_NVFP4_ERR_UNSUPPORTED, "too many rows (limit 2^26)");
  int dev, sms;
  if ((rc = moe::api_device(&dev, &sms))) return rc;
  if (T == 0) return MOE_NVFP4_OK;
  if ((rc = check_pointers(x_dev, q_dev, scales_dev))) return rc;
  if (!al(inv_dev, 4)) return moe::api_fail(MOE_NVFP4_ERR_INVALID_ARG, "inv must be 4-byte aligned");
  return done(moe::launch_fp8_quantize(static_cast<const uint16_t*>(x_dev), T, K, inv_dev, k,
                                       static_cast<uint8_t*>(q_dev), scales_dev, static_cast<cudaStream_t>(stream)),
              "fp8 quantize");
}

int moe_nvfp4_fp8_swiglu_quantize(const void* gu_dev, int64_t R, int32_t I, void* q_dev, float* scales_dev,
                                  void* stream) {
  int rc = check_rows(R, "R is negative");
  if (rc || (rc = check_width(I, "I"))) return rc;
  int dev, sms;
  if ((rc = moe::api_device(&dev, &sms))) return rc;
  if (R == 0) return MOE_NVFP4_OK;
  if ((rc = check_pointers(gu_dev, q_dev, scales_dev))) return rc;
  return done(moe::launch_fp8_swiglu_quantize(static_cast<const uint16_t*>(gu_dev), R, I, static_cast<uint8_t*>(q_dev),
                                              scales_dev, static_cast<cudaStream_t>(stream)),
              "fp8 SwiGLU quantize");
}

int moe_nvfp4_fp8_quantize_weights(const void* w_dev, int64_t n, int32_t N, int32_t K, void* q_dev, float* scales_dev,
                                   void* stream) {
  int rc = check_rows(n, "n is negative");
  if (rc || (rc = check_width(K, "K"))) return rc;
  if (N < 1 || N > 1 << 20) return bad("N outside 1..1048576", N);
  if (n > 65535) return moe::api_fail(MOE_NVFP4_ERR_UNSUPPORTED, "more than 65535 weights in one call");
  int dev, sms;
  if ((rc = moe::api_device(&dev, &sms))) return rc;
  if (n == 0) return MOE_NVFP4_OK;
  if ((rc = check_pointers(w_dev, q_dev, scales_dev))) return rc;
  return done(moe::launch_fp8_quantize_weights(static_cast<const uint16_t*>(w_dev), n, N, K,
                                               static_cast<uint8_t*>(q_dev), scales_dev,
                                               static_cast<cudaStream_t>(stream)),
              "fp8 quantize weights");
}

int moe_nvfp4_fp8_matmul(const void* a_dev, const float* a_scales_dev, int64_t M, const void* b_dev,
                         const float* b_scales_dev, int32_t E, int32_t N, int32_t K, const int32_t* offsets_dev,
                         void* out_dev, int32_t out_type, void* stream) {
  int rc = check_rows(M, "M is negative");
  if (rc || (rc = check_width(K, "K"))) return rc;
  if (E < 1 || E > 1024) return moe::api_fail(MOE_NVFP4_ERR_UNSUPPORTED, "E outside 1..1024");
  if (!offsets_dev && E != 1) return bad("E must be 1 without offsets", E);
  if (N < 8 || N % 8 || N > kMaxWidth)
    return moe::api_fail(MOE_NVFP4_ERR_UNSUPPORTED, "N must be a multiple of 8 in 8..65536");
  if (out_type != MOE_NVFP4_FP8_OUT_BF16 && out_type != MOE_NVFP4_FP8_OUT_F32) return bad("out_type unknown", out_type);
  moe::Fp8Tile forced;
  if ((rc = check_tile(&forced))) return rc;
  int dev, sms;
  if ((rc = moe::api_device(&dev, &sms))) return rc;
  if (M == 0) return MOE_NVFP4_OK;
  if ((rc = check_pointers(a_dev, out_dev, a_scales_dev)) || (rc = check_pointers(b_dev, out_dev, b_scales_dev)))
    return rc;
  if (!al(offsets_dev, 4)) return moe::api_fail(MOE_NVFP4_ERR_INVALID_ARG, "offsets must be 4-byte aligned");
  moe::Fp8Matmul p{};
  p.a = static_cast<const uint8_t*>(a_dev);
  p.a_scales = a_scales_dev;
  p.b = static_cast<const uint8_t*>(b_dev);
  p.b_scales = b_scales_dev;
  p.offsets = offsets_dev;
  p.M = M;
  p.E = E;
  p.N = N;
  p.K = K;
  p.out = out_dev;
  p.out_f32 = out_type == MOE_NVFP4_FP8_OUT_F32;
  return done(moe::launch_fp8_matmul(p, forced, dev, sms, static_cast<cudaStream_t>(stream)), "fp8 matmul");
}

}  // extern "C"
