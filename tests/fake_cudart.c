/* Stands in front of the CUDA runtime in a process without a GPU: the calls that
 * plan and launch a kernel succeed, or fail where the test says so, and are
 * counted.  Only what the tests of test_host_launches.py reach is here. */
#include <stddef.h>

enum { kFails = 2 }; /* cudaErrorMemoryAllocation */
static int calls, fail_at, launches, failed_launch;
static unsigned grids[64][6];

void fake_reset(int at) { calls = launches = failed_launch = 0, fail_at = at; }
int fake_calls(void) { return calls; }
int fake_launches(void) { return launches; }
int fake_failed_launch(void) { return failed_launch; }
unsigned fake_grid(int launch, int axis) { return grids[launch][axis]; }

static int next(void) { return ++calls == fail_at ? kFails : 0; }

int cudaGetDevice(int* device) {
  *device = 0;
  return next();
}
int cudaDeviceGetAttribute(int* value, int attribute, int device) {
  (void)attribute, (void)device;
  *value = 152; /* asked for the number of SMs alone */
  return 0;
}
int cudaFuncSetAttribute(const void* fn, int attribute, int value) {
  (void)fn, (void)attribute, (void)value;
  return next();
}
int cudaOccupancyMaxActiveClusters(int* n, const void* fn, const void* config) {
  (void)fn;
  /* (a grid of 64 clusters is asked about) */
  *n = 144 / (int)(*(const unsigned*)config / 64);
  return next();
}
int cudaLaunchKernelExC(const void* config, const void* fn, void** args) {
  (void)fn, (void)args;
  const unsigned* grid = config; /* the configuration begins with the grid and the block */
  const int rc = next();
  failed_launch |= rc != 0;
  if (rc == 0 && launches < 64) {
    for (int i = 0; i < 6; ++i) grids[launches][i] = grid[i];
    ++launches;
  }
  return rc;
}
int cudaGetLastError(void) { return 0; }
