// Argument-check macro of the ABI layer.
#pragma once

#include "common.h"

#define REQUIRE(cond, code, ...)   \
  do {                             \
    if (!(cond)) {                 \
      lq::set_error(__VA_ARGS__);  \
      return (code);               \
    }                              \
  } while (0)
