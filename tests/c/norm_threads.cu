// dpo_norm_forward and dpo_norm_backward from several host threads at once, each on its own stream and
// buffers, at lengths that use the same kernels with different amounts of shared memory: every call
// must succeed. Prints "ok" or the number of calls that failed.
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>

#include <cuda_runtime.h>

#include "dpo.h"

int main() {
  const int rows = 2400, calls = 6000;
  const int lengths[] = {1800, 2048, 1808, 2040, 1816, 2032};
  std::atomic<int> failed{0}, ready{0};
  std::vector<std::thread> threads;
  const int n = sizeof(lengths) / sizeof(lengths[0]);
  for (int i = 0; i < n; ++i)
    threads.emplace_back([&, i] {
      const int d = lengths[i];
      cudaStream_t st;
      void *x = nullptr, *y = nullptr, *dx = nullptr, *ws = nullptr;
      float *rstd = nullptr, *dw = nullptr;
      size_t bytes = 0;
      const size_t cells = static_cast<size_t>(rows) * d * 2;
      if (cudaStreamCreate(&st) != cudaSuccess || dpo_norm_workspace_size(rows, d, &bytes) != DPO_OK ||
          cudaMalloc(&x, cells) != cudaSuccess || cudaMalloc(&y, cells) != cudaSuccess ||
          cudaMalloc(&dx, cells) != cudaSuccess || cudaMalloc(&ws, bytes) != cudaSuccess ||
          cudaMalloc(&rstd, sizeof(float) * rows) != cudaSuccess ||
          cudaMalloc(&dw, sizeof(float) * d) != cudaSuccess ||
          cudaMemsetAsync(x, 0, cells, st) != cudaSuccess) {
        failed += 1000000;
        ready += 1;
        return;
      }
      dpo_norm norm = {};
      norm.kind = DPO_NORM_RMS;
      norm.dtype = norm.weight_dtype = DPO_BF16;
      norm.rows = rows;
      norm.d = d;
      norm.eps = 1e-5f;
      norm.x = x;
      norm.x_stride = d;
      dpo_norm_grads g = {};
      g.rstd = rstd;
      g.dy = y;
      g.dy_dtype = DPO_BF16;
      g.dy_stride = d;
      g.dx = dx;
      g.dx_stride = d;
      g.dweight = dw;
      cudaStreamSynchronize(st);
      ready += 1;
      while (ready.load() < n) std::this_thread::yield();
      for (int k = 0; k < calls; ++k) {
        if (dpo_norm_forward(&norm, y, d, nullptr, rstd, nullptr, st) != DPO_OK) ++failed;
        if (dpo_norm_backward(&norm, &g, ws, bytes, st) != DPO_OK) ++failed;
        if (k % 100 == 99) cudaStreamSynchronize(st);
      }
      if (cudaStreamSynchronize(st) != cudaSuccess) ++failed;
    });
  for (auto& t : threads) t.join();
  if (failed.load() == 0) std::puts("ok");
  else std::printf("%d calls failed\n", failed.load());
  return failed.load() != 0;
}
