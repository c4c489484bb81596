/* Test-only stand-in of libpa.so's calls that _binding makes: each waits, two seconds at
 * most, for another thread to set `go`, and says whether that happened. */
#include <time.h>

volatile int go = 0;
volatile int waiting = 0;

static int wait_for_go(void) {
  struct timespec nap = {0, 1000000};
  waiting = 1;
  for (int i = 0; i < 2000 && !go; ++i) nanosleep(&nap, 0);
  return go ? 0 : -3;
}
int pa_rope_append(void) { return wait_for_go(); }
int pa_rope_append_fp4(void) { return wait_for_go(); }
int pa_gather_fp4(void) { return wait_for_go(); }
int pa_attention_varlen_fp4(void) { return wait_for_go(); }
