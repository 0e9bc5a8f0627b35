// Calls of the library's launches with copies that are waited for beyond what they
// bring, so that the kernels' bounded waits run out.
#include <cuda_runtime.h>

#include "moe_internal.h"

extern "C" int lost_project(int T, int K, int N, int group, int sms, int lost, const void* x, const void* w, void* y) {
  moe::ProjectParams p = {};
  p.T = T, p.K = K, p.N = N, p.group = group, p.sms = sms, p.lost = lost;
  p.y_dtype = 0;
  p.x_stride = K, p.y_stride = N, p.w_stride = (K / 2 + K / group * 2 + 15) / 16 * 16;
  p.x = static_cast<const uint16_t*>(x);
  p.w = static_cast<const uint8_t*>(w);
  p.y = y;
  return moe::launch_project(p, nullptr);
}

// Cache [pages][page_size][Hkv][D] and out of bf16, one row a sequence.
extern "C" int lost_attend(int B, int Hq, int Hkv, int D, int page_size, int pages, int max_pages, int sms, int lost,
                           const void* q, const void* k, const void* v, const int* table, const int* lens,
                           const int* q_start, void* out, float* lse, void* ws) {
  moe::AttendParams p = {};
  p.T = p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.D = D, p.sms = sms, p.lost = lost;
  p.out_dtype = 1;
  p.page_size = page_size, p.pages = pages, p.max_pages = max_pages;
  p.scale = 0.125f;
  p.q_stride = p.o_stride = Hq * D, p.q_head = p.o_head = p.kc_head = p.vc_head = D;
  p.kc_slot = p.vc_slot = Hkv * D, p.kc_page = p.vc_page = (long long)page_size * Hkv * D;
  p.table_stride = max_pages;
  p.q = static_cast<const uint16_t*>(q), p.k = static_cast<const uint16_t*>(k), p.v = static_cast<const uint16_t*>(v);
  p.table = table, p.lens = lens, p.q_start = q_start;
  p.out = out, p.lse = lse, p.ws = ws;
  return moe::launch_attend(p, nullptr);
}
